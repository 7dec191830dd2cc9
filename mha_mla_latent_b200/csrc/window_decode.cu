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
// with the 16 (or all) heads it concerns only.  O^T needs 32 columns per 128 latent columns, so
// two streams of tiles (even and odd, one softmax group each) keep an accumulator of their own
// and the chain load -> S -> softmax -> O of one overlaps the other's.  The streams' results are
// merged in tensor memory when a piece (part of one sequence) ends.
//
// What bounds it is HBM: the cached rows of the visible tokens, read once.  The products take
// about a third of that time at d_c = 256 and the softmax a tenth.
//
// The running maximum is raised lazily: a thread that sees a score above m[h] + kTau reports it
// in the group's per-tile barrier (an OR over its 128 threads) and the group then takes the
// tile's maxima, rescales its accumulator and goes on.  Between raises P stays below 2^kTau.
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer, warps 2-3 dequantise a quantised latent,
// warps 4-7 and 8-11 the softmax groups.  Every wait is bounded; a group leaves its loop only
// where all of it does (the barrier carries the failure too).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "decode_common.cuh"
#include "sm100.cuh"

namespace mla {
namespace wdec {

using namespace sm100;

constexpr int kUnit = 64;                 // tokens of a schedule tile and of a TMA box
constexpr int kT = 128;                   // tokens per product tile: two units
constexpr uint32_t kHalf = kUnit * 128;   // bytes of a box: 64 rows x 128 B
constexpr uint32_t kSlot = 2 * kHalf;     // ring slot: 128 tokens x 64 columns
constexpr int kThreads = 384;
constexpr float kTau = 8.0f;              // lazy-rescale threshold, log2 units
constexpr uint32_t kCols = 256, kSCol = 0, kOCol = 64;   // S: 2 x 32 columns, O: 2 streams x 2 blocks x 32
constexpr uint32_t kSmemMax = 232448;
constexpr int kMaxC = 4, kMaxK = 8, kMaxRaw = 3;

struct Args {
  int H, G, d_c, dcp, R, P, T_cap;
  int n_cbox, n_kbox, kr_rows;            // boxes per token row; heads a key box is multiplied with
  int NC, NK, NRAW;                       // latent tiles, key boxes, code tiles in the rings
  MlaWindow win;
  Sched sched;
  const int32_t* seq_lens;
  const float* qrope;                     // [B][H][8], rotated, scaled
  float* opart;                           // [P][H][d_c]
  float* mlpart;                          // [H][P][2]
  const __half* scales;
  uint32_t code_row;
  mla_cache_t cache;
  int32_t* err;
  uint64_t wait_ns;
  uint32_t off_q, off_qr, off_p, off_c, off_k, off_raw, raw_stage, off_red, off_bar;
};

enum {
  kCFull = 0, kCEmpty = kCFull + kMaxC, kKFull = kCEmpty + kMaxC, kKEmpty = kKFull + kMaxK, kRFull = kKEmpty + kMaxK,
  kREmpty = kRFull + kMaxRaw, kSFull = kREmpty + kMaxRaw, kSEmpty = kSFull + 2, kPFull = kSEmpty + 2, kODone = kPFull + 2,
  kOEmpty = kODone + 2, kQFull, kQEmpty, kMeet, kDone, kBars
};
// Exchange area, floats: per group the tile maxima of its warps [2][4][32]; by piece parity the
// sums of all warps [2][2][4][32] and the groups' maxima [2][2][32].
constexpr uint32_t kRedBytes = (2 * 4 * 32 + 2 * 2 * 4 * 32 + 2 * 2 * 32) * 4;

__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)r * 128u + (uint32_t)(((c ^ r) & 7) << 4); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Walk over a worker's pieces in tiles: x is the tile's first token in the sequence's span.
struct Walk {
  const Args* a;
  int pc, end, b, x, x0, x1;
  Span span;
  __device__ void init(const Args* args, int w) {
    a = args;
    pc = a->sched.worker_first[w];
    end = a->sched.worker_first[w + 1];
    if (pc < end) load();
  }
  __device__ void load() {
    b = a->sched.piece_b[pc]; x0 = a->sched.piece_t0[pc]; x1 = a->sched.piece_t1[pc]; x = x0;
    span = unit_span(__ldg(a->seq_lens + b), 1, kUnit, a->win);
  }
  __device__ bool valid() const { return pc < end; }
  __device__ bool first() const { return x == x0; }
  __device__ bool last() const { return x + kT >= x1; }
  __device__ int rows() const { return min(kT, x1 - x); }
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

// N: heads padded to 16 or 32; QB: code width of a quantised latent (4 or 2), 0 for bf16.
template <int N, int QB>
__global__ void __launch_bounds__(kThreads, 1)
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

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kBars; ++i) {
      int n = 1;
      if (i >= kCFull && i < kCEmpty && QB) n = 2;      // both dequantising warps
      if (i >= kREmpty && i < kSFull) n = 2;
      if (i >= kSEmpty && i < kODone) n = 4;            // a softmax group's warps (S read, P written)
      if (i == kOEmpty || i == kMeet) n = 8;            // both groups
      if (i == kQFull) n = 2;                           // Q_lat bytes, the RoPE rows
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
  }
  // query rows past the last head and the zero blocks of the RoPE operand stay zero
  for (uint32_t i = threadIdx.x; i < (a.off_p - a.off_q) / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + a.off_q)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_c);
    tma_prefetch_desc(&tm_kr);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const uint32_t c_bytes = (uint32_t)a.n_cbox * kSlot;
  pdl_wait();   // schedule, absorbed queries and the cache come from earlier kernels
  pdl_trigger();
  const int w = blockIdx.x;

  if (warp == 0) {
    // ============================================================ TMA producer (lane 0)
    if (lane == 0) {
      // cursors: latent (or code) tiles with the queries, and key boxes, whose slots free up at
      // different times
      Walk wc, wk;
      wc.init(&a, w);
      wk = wc;
      int nc = 0, nk = 0, kb = 0, tk = 0, u = 0;
      int looks = 0;
      uint64_t idle = 0;
      auto row_of = [&](const Walk& it, int unit) {
        const MlaLoc lc = mla_loc(a.cache, it.b, it.token(unit), a.err);   // a unit lies in one block
        return lc.pb * lc.cap + lc.pt;
      };
      while (wc.valid() || wk.valid()) {
        bool progress = false;
        if (wc.valid()) {
          const int s = QB ? nc % NRAW : nc % NC, ring = QB ? NRAW : NC;
          const bool q_ok = !wc.first() || u == 0 || mbar_test(bar(kQEmpty), (u - 1) & 1);
          if (q_ok && (nc < ring || mbar_test(bar((QB ? kREmpty : kCEmpty) + s), ((nc / ring) - 1) & 1))) {
            if (wc.first()) {
              mbar_expect_tx(bar(kQFull), (uint32_t)a.n_cbox * a.H * 128u);
              for (int k = 0; k < a.n_cbox; ++k)
                tma_load_2d(sb + a.off_q + k * N * 128, &tm_q, bar(kQFull), k * 64, wc.b * a.H);
              ++u;
            }
            const int units = wc.units();
            if (QB) mbar_expect_tx(bar(kRFull + s), (uint32_t)units * kUnit * a.code_row);
            else mbar_expect_tx(bar(kCFull + s), (uint32_t)units * a.n_cbox * kHalf);
            for (int j = 0; j < units; ++j) {
              const int row = row_of(wc, j);
              if (QB) {
                tma_load_2d(sb + a.off_raw + s * a.raw_stage + j * kUnit * a.code_row, &tm_c, bar(kRFull + s), 0, row);
              } else {
                for (int k = 0; k < a.n_cbox; ++k)
                  tma_load_2d(sb + a.off_c + s * c_bytes + k * kSlot + j * kHalf, &tm_c, bar(kCFull + s), k * 64, row);
              }
            }
            wc.next();
            ++nc;
            progress = true;
          }
        }
        if (wk.valid() && tk < nc) {   // keys never run ahead of their tile's latent copy
          const int s = nk % NK;
          if (nk < NK || mbar_test(bar(kKEmpty + s), ((nk / NK) - 1) & 1)) {
            const int units = wk.units();
            mbar_expect_tx(bar(kKFull + s), (uint32_t)units * kHalf);
            for (int j = 0; j < units; ++j)
              tma_load_2d(sb + a.off_k + s * kSlot + j * kHalf, &tm_kr, bar(kKFull + s), kb * 64, row_of(wk, j));
            ++nk;
            if (++kb == a.n_kbox) { kb = 0; ++tk; wk.next(); }
            progress = true;
          }
        }
        if (progress) {
          looks = 0;
        } else if ((++looks & 63) == 0) {
          const uint64_t now = globaltimer();
          if (looks == 64) idle = now;
          if (*abort_flag || now - idle > lim) { *abort_flag = 1; break; }
        }
      }
      // every issued copy lands before the CTA exits
      volatile int never = 0;
      auto drain = [&](int first, int ring, int issued) {
        for (int i = max(0, issued - ring); i < issued; ++i) mbar_spin(bar(first + i % ring), (i / ring) & 1, &never, lim);
      };
      drain(QB ? kRFull : kCFull, QB ? NRAW : NC, nc);
      drain(kKFull, NK, nk);
      if (*abort_flag && u > 0) {   // the queries' copy (its barrier may still miss the RoPE rows: wait a moment instead)
        const uint64_t t0 = globaltimer();
        while (!mbar_test(bar(kQFull), (u - 1) & 1) && globaltimer() - t0 < 1000000ull) {}
      }
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer (converged warp, elected lane)
    const uint32_t id_s = idesc_bf16_f32(kT, N, false, false), id_k = idesc_bf16_f32(kT, a.kr_rows, false, false);
    const uint32_t id_o = idesc_bf16_f32(kT, N, true, true);
    const uint64_t desc_q = smem_desc(sb + a.off_q, 16, 1024, kLayoutSW128);
    const uint64_t desc_qr = smem_desc(sb + a.off_qr, 16, 1024, kLayoutSW128);
    auto ready = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_test(bar(i), parity)) != 0; };
    const int n_blk = (a.dcp + 127) / 128;   // blocks of 128 latent columns
    Walk i1, i2;                             // tiles whose S, and whose O, is issued next
    i1.init(&a, w);
    i2 = i1;
    int n1 = 0, j1 = 0, nk = 0, n2 = 0, u1 = 0, u2 = 0;   // j1: parts of S(n1) issued (latent, then key boxes)
    bool ok = true;
    int looks = 0;
    uint64_t idle = 0;
    while (ok && i2.valid()) {
      bool progress = false;
      if (i1.valid()) {
        const int s = n1 & 1;
        if (j1 == 0) {
          if ((n1 < 2 || ready(kSEmpty + s, ((n1 >> 1) - 1) & 1)) && (!i1.first() || ready(kQFull, u1 & 1)) &&
              ready(kCFull + n1 % NC, (n1 / NC) & 1)) {
            tc_fence_after();
            if (elect_one()) {
              uint64_t da = smem_desc(sb + a.off_c + (n1 % NC) * c_bytes, 16, 1024, kLayoutSW128), db = desc_q;
              const uint32_t d = tmem + kSCol + s * 32;
              for (int k = 0; k < a.n_cbox; ++k) {   // a box of 64 columns is four steps
                tc_mma_bf16(d, da, db, id_s, k > 0);
                tc_mma_bf16(d, da + 2, db + 2, id_s, 1);
                tc_mma_bf16(d, da + 4, db + 4, id_s, 1);
                tc_mma_bf16(d, da + 6, db + 6, id_s, 1);
                da += kSlot >> 4;
                db += (N * 128) >> 4;
              }
            }
            __syncwarp();
            j1 = 1;
            progress = true;
          }
        } else if (ready(kKFull + nk % NK, (nk / NK) & 1)) {
          tc_fence_after();
          const int kb = j1 - 1;
          const bool done = j1 == a.n_kbox;
          if (elect_one()) {
            // KV heads 8 kb .. 8 kb + 7: query heads from col on
            const int col = a.kr_rows == N ? 0 : (kb * 8 * a.G) & ~15;
            const uint32_t d = tmem + kSCol + s * 32 + col;
            const uint64_t da = smem_desc(sb + a.off_k + (nk % NK) * kSlot, 16, 1024, kLayoutSW128);
            const uint64_t db = desc_qr + (uint32_t)kb * (a.kr_rows * 128u >> 4);
            const int steps = min(4, (a.R - kb * 64 + 15) / 16);
            for (int k = 0; k < steps; ++k) tc_mma_bf16(d, da + 2 * k, db + 2 * k, id_k, 1);
            tc_commit(bar(kKEmpty + nk % NK));
            if (done) {
              tc_commit(bar(kSFull + s));
              if (i1.last()) tc_commit(bar(kQEmpty));
            }
          }
          __syncwarp();
          ++nk;
          ++j1;
          if (done) {
            j1 = 0;
            if (i1.last()) ++u1;
            i1.next();
            ++n1;
          }
          progress = true;
        }
      }
      // O(n2): its P, and for a stream's first tile of a piece the accumulators read out
      if (n2 < n1 && ready(kPFull + (n2 & 1), (n2 >> 1) & 1)) {
        const bool fresh = i2.x - i2.x0 < 2 * kT;   // the piece's first or second tile: its stream starts
        if (!fresh || u2 == 0 || ready(kOEmpty, (u2 - 1) & 1)) {
          tc_fence_after();
          const int s = n2 & 1;
          if (elect_one()) {
            const uint64_t dp = smem_desc(sb + a.off_p + s * kPBytes, 16, 8 * kPRow, kPLayout);
            const uint64_t dc = smem_desc(sb + a.off_c + (n2 % NC) * c_bytes, kSlot, 1024, kLayoutSW128);
            const int steps = (i2.rows() + 15) / 16;
            for (int m = 0; m < n_blk; ++m)
              for (int k = 0; k < steps; ++k)
                tc_mma_bf16(tmem + kOCol + s * 64 + m * 32, dc + (uint32_t)m * (2 * kSlot >> 4) + 128u * k,
                            dp + (uint32_t)k * (16 * kPRow >> 4), id_o, !fresh || k > 0);
            tc_commit(bar(kCEmpty + n2 % NC));
            tc_commit(bar(kODone + s));
          }
          __syncwarp();
          if (i2.last()) ++u2;
          i2.next();
          ++n2;
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
  } else if (warp < 4) {
    // ============================================================ dequantisation (two token rows per thread)
    if (QB != 0) {
      const int t = (warp - 2) * 32 + lane;   // rows t and t + 64 of each tile
      Walk it;
      it.init(&a, w);
      bool ok = true;
      for (int n = 0; ok && it.valid(); ++n, it.next()) {
        const int rs = n % NRAW, cs = n % NC;
        const int L = __ldg(a.seq_lens + it.b);
        // where the rows' scales (and ring rows) come from, asked for ahead of the waits
        const __half* sp[2];
        bool live[2], ring[2];
        size_t slot[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = t + 64 * j;
          live[j] = it.visible(r);
          ring[j] = false;
          sp[j] = a.scales;
          slot[j] = 0;
          if (live[j]) {
            const int tp = it.token(j) + t;
            const MlaLoc lc = mla_loc(a.cache, it.b, it.token(j), a.err);
            sp[j] = a.scales + ((size_t)lc.pb * lc.cap + lc.pt + t) * (a.d_c / 32);
            if (a.cache.c_resid && tp >= L - MLA_RESID_WINDOW) {
              slot[j] = (size_t)it.b * MLA_RESID_WINDOW + (tp & (MLA_RESID_WINDOW - 1));
              ring[j] = __ldg(a.cache.resid_pos + slot[j]) == tp;
            }
          }
        }
        __half sc[2][8];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) sc[j][k] = k < a.d_c / 32 && live[j] ? __ldg(sp[j] + k) : __float2half(0.f);
        ok = __all_sync(0xffffffffu, mbar_spin(bar(kRFull + rs), (n / NRAW) & 1, abort_flag, lim));
        if (ok && n >= NC) ok = __all_sync(0xffffffffu, mbar_spin(bar(kCEmpty + cs), ((n / NC) - 1) & 1, abort_flag, lim));
        if (!ok) break;
        uint8_t* C = smem + a.off_c + cs * c_bytes;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = t + 64 * j;
          auto put = [&](int chunk, uint4 v) { *reinterpret_cast<uint4*>(C + (chunk >> 3) * kSlot + sw128(r, chunk)) = v; };
          if (ring[j]) {   // one of the window's unquantised tokens
            const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.cache.c_resid) + slot[j] * a.d_c);
            for (int c = 0; c < a.d_c / 8; ++c) put(c, __ldg(src + c));
          } else if (live[j]) {
            const uint8_t* codes = smem + a.off_raw + rs * a.raw_stage + r * a.code_row;
#pragma unroll 1
            for (int g = 0; g < a.d_c / 32; ++g) {
              __half hs = sc[j][0];
#pragma unroll
              for (int k = 1; k < 8; ++k) hs = g == k ? sc[j][k] : hs;
              const float sv = __half2float(hs);
              uint32_t wd[4];
              if (QB == 4) {
                const uint4 cw = *reinterpret_cast<const uint4*>(codes + g * 16);
                wd[0] = cw.x; wd[1] = cw.y; wd[2] = cw.z; wd[3] = cw.w;
              } else {
                const uint2 cw = *reinterpret_cast<const uint2*>(codes + g * 8);
                wd[0] = cw.x; wd[1] = cw.x >> 16; wd[2] = cw.y; wd[3] = cw.y >> 16;
              }
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                // offset codes in the mantissa of 2^23: the float exceeds the base by the code;
                // code x scale is rounded to bf16, the products' operand type
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t f = wd[ch] >> (2 * QB * e);
                  constexpr uint32_t top = 1u << (QB ? QB - 1 : 0), mask = 2 * top - 1;
                  const float base = 8388608.0f + (float)top;
                  const float lo = __uint_as_float(0x4B000000u | ((f ^ top) & mask)) - base;
                  const float hi = __uint_as_float(0x4B000000u | (((f >> QB) ^ top) & mask)) - base;
                  o[e] = pack2(lo * sv, hi * sv);
                }
                put(4 * g + ch, make_uint4(o[0], o[1], o[2], o[3]));
              }
            }
          } else {
            for (int c = 0; c < a.d_c / 8; ++c) put(c, make_uint4(0, 0, 0, 0));
          }
          for (int c = a.d_c / 8; c < a.dcp / 8; ++c) put(c, make_uint4(0, 0, 0, 0));   // padding columns
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kREmpty + rs));
          mbar_arrive(bar(kCFull + cs));
        }
      }
    }
  } else {
    // ============================================================ softmax groups
    const int s = warp >= 8;                 // stream
    const int q = warp & 3, r = 32 * q + lane;
    const uint32_t lane0 = tmem + ((uint32_t)(32 * q) << 16);
    float* red = reinterpret_cast<float*>(smem + a.off_red) + s * 4 * 32;
    float* sums = reinterpret_cast<float*>(smem + a.off_red) + 2 * 4 * 32;   // [parity][stream][warp][32]
    float* tops = sums + 2 * 2 * 4 * 32;                                     // [parity][stream][32]
    auto warp_wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_spin(bar(i), parity, abort_flag, lim)) != 0; };
    auto arrive = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    Walk it;
    it.init(&a, w);
    int n = 0, u = 0;                        // tiles and pieces of the CTA
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
            const float4 x = __ldg(src), y = __ldg(src + 1);
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
        if (!fail) fail = !warp_wait(kSFull + s, k & 1);
        float x[N];
        {
          uint32_t raw[N];
          tc_fence_after();
          tmem_ld<N>(lane0 + kSCol + s * 32, raw);
          tmem_wait_ld();
          const bool vis = it.visible(r);
#pragma unroll
          for (int h = 0; h < N; ++h) {
            asm volatile("" : "+r"(raw[h]));   // the values exist only after the wait
            x[h] = vis ? __uint_as_float(raw[h]) : -INFINITY;
          }
        }
        tc_fence_before();
        arrive(kSEmpty + s);
        bool raise = !some;
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
            const bool up = t > m[h] + (some ? kTau : 0.f) || !some;
            al[h] = up ? exp2f(m[h] - t) : 1.f;   // m = -inf: 0
            m[h] = up ? t : m[h];
            l[h] = some ? l[h] * al[h] : 0.f;
          }
          if (some) {
            for (int blk = 0; blk < (a.dcp + 127) / 128; ++blk) {
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
        // P row of this token, rounded to bf16 (the product's operand type)
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
          uint8_t* C = smem + a.off_c + (n % NC) * c_bytes;
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
        if (!fail && done0 > 0) fail = !warp_wait(kODone, (done0 - 1) & 1);
        if (!fail && done1 > 0) fail = !warp_wait(kODone + 1, (done1 - 1) & 1);
        if (group_or(1 + s, fail)) break;
        tc_fence_after();
        // this group writes heads [N/2 s, N/2 s + N/2): lane = latent column
        const float* t0 = tops + par * 2 * 32;
        const float* l0 = sums + par * 2 * 4 * 32;
        constexpr int HN = N / 2;
        for (int blk = 0; blk < (a.dcp + 127) / 128; ++blk) {
          const int c = blk * 128 + r;
          for (int h0 = 0; h0 < HN; h0 += 8) {
            uint32_t o0[8], o1[8];
            tmem_ld8(lane0 + kOCol + blk * 32 + HN * s + h0, o0);
            tmem_ld8(lane0 + kOCol + 64 + blk * 32 + HN * s + h0, o1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              asm volatile("" : "+r"(o0[e]), "+r"(o1[e]));
              const int h = HN * s + h0 + e;
              const float m0 = t0[h], m1 = t0[32 + h], M = fmaxf(m0, m1);
              // a stream without a tile in this piece holds nothing (its columns are stale)
              const float v0 = m0 == -INFINITY ? 0.f : exp2f(m0 - M) * __uint_as_float(o0[e]);
              const float v1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M) * __uint_as_float(o1[e]);
              if (h < a.H && c < a.d_c) a.opart[((size_t)it.pc * a.H + h) * a.d_c + c] = v0 + v1;
            }
          }
        }
        if (s == 0 && r < a.H) {
          const float m0 = t0[r], m1 = t0[32 + r], M = fmaxf(m0, m1);
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum0 += l0[k * 32 + r];
            sum1 += l0[(4 + k) * 32 + r];
          }
          a.mlpart[((size_t)r * a.P + it.pc) * 2] = M;
          a.mlpart[((size_t)r * a.P + it.pc) * 2 + 1] =
              (m0 == -INFINITY ? 0.f : exp2f(m0 - M) * sum0) + (m1 == -INFINITY ? 0.f : exp2f(m1 - M) * sum1);
        }
        tc_fence_before();
        arrive(kOEmpty);
        ++u;
      }
      it.next();
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
  uint32_t off_q, off_qr, off_p, off_c, off_k, off_raw, raw_stage, off_red, off_bar, total;
};

// [Q_lat boxes][RoPE query boxes][P of two streams][latent ring][key-box ring][code ring]
// [exchange][barriers].  The slots left (16 KB: 128 tokens x 64 columns) go to latent tiles and
// key boxes in the proportion a tile needs them, at least two latent tiles (one per stream).
static bool layout(const mla_config_t& c, int R, Layout* out) {
  Layout L{};
  const int G = c.n_heads / c.n_kv_heads, qbits = mla_kind_quant(c.cache_kind) ? mla_quant_bits(c.cache_kind) : 0;
  L.N = c.n_heads <= 16 ? 16 : 32;
  L.n_cbox = (c.d_c + 63) / 64;
  L.n_kbox = (R + 63) / 64;
  L.kr_rows = L.n_kbox == 1 || G > 2 ? L.N : 16;
  L.NRAW = qbits ? 2 : 0;
  L.raw_stage = (uint32_t)(kT * c.d_c * qbits / 8);
  L.off_qr = (uint32_t)(L.n_cbox * L.N) * 128;
  L.off_p = L.off_qr + (uint32_t)(L.n_kbox * L.kr_rows) * 128;
  L.off_c = L.off_p + 2u * kT * L.N * 2;
  const uint32_t tail = kRedBytes + 8 * kBars + 16 + 1024;
  const uint32_t fixed = L.off_c + L.NRAW * L.raw_stage + tail;
  if (fixed > kSmemMax) return false;
  const int slots = (int)((kSmemMax - fixed) / kSlot);
  const int per = L.n_cbox + L.n_kbox;
  L.NC = std::max(2, std::min(kMaxC, (slots + per - 1) / per));
  L.NK = std::min(kMaxK, slots - L.NC * L.n_cbox);
  if (L.NK < 1 && L.NC > 2) {
    L.NC = 2;
    L.NK = std::min(kMaxK, slots - L.NC * L.n_cbox);
  }
  if (L.NK < 1) return false;
  L.off_k = L.off_c + (uint32_t)(L.NC * L.n_cbox) * kSlot;
  L.off_raw = L.off_k + (uint32_t)L.NK * kSlot;
  L.off_red = L.off_raw + L.NRAW * L.raw_stage;
  L.off_bar = L.off_red + kRedBytes;
  L.total = L.off_bar + 8 * kBars + 16 + 1024;
  *out = L;
  return true;
}

}  // namespace wdec
}  // namespace mla

// Shapes: bf16 with r = 4 kept pairs per KV head, up to 32 query heads and 32 KV heads, d_c a
// multiple of 32 up to 256, code rows of whole 16 bytes, key rows of whole 16 bytes.
bool mla_window_decode_capable(const mla_plan& p) {
  const mla_config_t& c = p.cfg;
  if (c.dtype != MLA_BF16 || c.r_pairs != 4 || c.n_heads > 32 || c.d_c % 32 != 0 || c.d_c > 256) return false;
  if (mla_kind_quant(c.cache_kind) && c.d_c * mla_quant_bits(c.cache_kind) / 8 % 16 != 0) return false;
  mla::wdec::Layout L;
  return mla::wdec::layout(c, p.R, &L);
}

cudaError_t mla_launch_window_decode(const mla_plan& p, const mla_cache_t& c, const int32_t* seq_lens, int B,
                                     const Sched& sched, const void* qlat, const float* qrope, float* opart,
                                     float* mlpart, int P, int G, MlaWindow win, cudaStream_t s) {
  using namespace mla::wdec;
  const mla_config_t& cfg = p.cfg;
  const int qbits = mla_kind_quant(cfg.cache_kind) ? mla_quant_bits(cfg.cache_kind) : 0;
  Layout L;
  if (!layout(cfg, p.R, &L)) return cudaErrorInvalidValue;
  Args a;
  a.H = cfg.n_heads; a.G = a.H / cfg.n_kv_heads; a.d_c = cfg.d_c; a.dcp = L.n_cbox * 64; a.R = p.R; a.P = P;
  a.T_cap = c.T_cap; a.n_cbox = L.n_cbox; a.n_kbox = L.n_kbox; a.kr_rows = L.kr_rows;
  a.NC = L.NC; a.NK = L.NK; a.NRAW = L.NRAW;
  a.win = win; a.sched = sched; a.seq_lens = seq_lens; a.qrope = qrope; a.opart = opart; a.mlpart = mlpart;
  a.scales = (const __half*)c.c_scales; a.code_row = (uint32_t)(cfg.d_c * qbits / 8); a.cache = c; a.err = p.err;
  a.wait_ns = (uint64_t)p.opt_wait_us * 1000u;
  a.off_q = L.off_q; a.off_qr = L.off_qr; a.off_p = L.off_p; a.off_c = L.off_c; a.off_k = L.off_k; a.off_raw = L.off_raw;
  a.raw_stage = L.raw_stage; a.off_red = L.off_red; a.off_bar = L.off_bar;
  const uint64_t rows = mla_cache_rows(c);
  CUtensorMap tm_c, tm_kr, tm_q;
  bool ok = map_2d(&tm_kr, false, c.k_rope, p.R, rows, 64, kUnit) &&
            map_2d(&tm_q, false, qlat, cfg.d_c, (uint64_t)B * a.H, 64, a.H);
  ok = ok && (qbits ? map_2d(&tm_c, true, c.c_kv, a.code_row, rows, a.code_row, kUnit)
                    : map_2d(&tm_c, false, c.c_kv, cfg.d_c, rows, 64, kUnit));
  if (!ok) return cudaErrorInvalidValue;
  auto pick = [&](auto n) {
    constexpr int N = decltype(n)::value;
    return qbits == 4 ? window_decode_kernel<N, 4> : qbits == 2 ? window_decode_kernel<N, 2> : window_decode_kernel<N, 0>;
  };
  const auto kern = L.N == 16 ? pick(std::integral_constant<int, 16>()) : pick(std::integral_constant<int, 32>());
  cudaError_t e = mla_smem_limit((const void*)kern, L.total);
  if (e != cudaSuccess) return e;
  if ((e = mla_profile_event(p, kProfAttention, false, s)) != cudaSuccess) return e;
  e = mla_launch_kernel(kern, dim3(G), dim3(kThreads), L.total, s, p.opt_pdl, tm_c, tm_kr, tm_q, a);
  if (e != cudaSuccess) return e;
  return mla_profile_event(p, kProfAttention, true, s);
}
