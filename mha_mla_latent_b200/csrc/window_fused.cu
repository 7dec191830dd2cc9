// Windowed latent attention in one launch: each CTA takes a unit of up to 128 rows (the query
// heads of a few KV heads x a block of consecutive queries of one sequence) from the raw
// queries to the finished output.
//
// Paper notes "MHA2MLA" (ACL 2025), §关键设计: W_uk is absorbed into the query, the partial-RoPE
// term is scored apart, the probability-weighted latent goes through W_uv.  Per unit, rows
// r = (KV head, query head of its group, query), in tiles of 128 tokens:
//     Q_lat[r][c]  = scale sum_d q[r][d] W_ukF[g(r)][d][c]               K = d_h
//     S[r][t]      = sum_c Q_lat[r][c] C[t][c] + sum_j Q_rope[r][j] KR[t][j]   K = d_c + 16 per 2 KV heads
//     O[r][c]     += sum_t P[r][t] C[t][c],  P = 2^(S - m) on the visible tokens
//     out[r][d]    = sum_c O[r][c] / l[r] W_uv[g(r)][c][d]               K = d_c
// all on the 5th-generation tensor cores with M = 128.  Rows of few KV heads keep the RoPE
// product short (its query operand is block-diagonal over the unit's KV heads), make each
// weight slice serve many rows, and leave nothing to merge: no partials go through memory.
// The price is that every unit of a sequence reads the window again, which the L2 serves.
//
// Operands that the CTA itself makes stay in tensor memory: the queries, the probabilities
// (over the scores they came from) and the merged latent are A operands of their products
// there, so shared memory holds Q_lat, the RoPE queries and the ring of tiles only.
// Tensor memory columns: [0, 256) O, also the absorption's accumulator; [256, 384) and
// [384, 512) S of even and odd tiles, also q, the merged latent's high halves and the output.
//
// Roles: warp 0 TMA producer (W_uk slices, tiles, W_uv slices through one ring), warp 1 MMA
// issuer, warps 4-11 the rows, two threads per row (queries, softmax, epilogue), warps 12-15 with
// a quantised latent the dequantisation, straight from the cache into the ring.  Every wait is
// bounded; waits poll without the suspended form, whose wake-up costs more than it frees here
// (each scheduler holds two row warps and at most one of the others).
//
// Bound by the tensor cores once the tiles flow (10 tiles of 128 tokens at d_c = 256 take 1.4 to
// 1.8 us each, some 85% of the measured dense rate) and by the latency of its ends: about 6 us
// from the launch to the first scores and 5 us from the last tile to the stored rows.  B200, 8
// sequences x 64 queries, 32 KV heads, window 1024, d_c = 256: 34.1 us; 4-bit latent 52 us, where
// a tile's conversion (a thread per row, about 3 us) bounds it, and 33 us at d_c = 128.  The
// head-row units with their absorption and merge launches take 179, 202 and 157 us there.
#include <cuda.h>

#include "decode_common.cuh"
#include "sm100.cuh"

namespace mla {
namespace fused {

using namespace sm100;

constexpr int kT = 128;               // tokens per tile
constexpr int kRows = 128;            // rows per unit
template <int QB> constexpr int kThreadsOf = QB ? 512 : 384;   // a quantised latent: a warpgroup that dequantises
constexpr uint32_t kBox = kT * 128;   // bytes of 128 rows x 64 bf16 columns
constexpr uint32_t kKrTile = kT * 64; // RoPE keys of a tile: 32 columns (4 KV heads)
constexpr int kMaxG = 4;              // KV heads per unit
constexpr float kTau = 8.0f;          // lazy-rescale threshold, log2 units
constexpr uint32_t kCols = 512, kOCol = 0, kSCol = 256;
constexpr uint32_t kSmemMax = 232448;

struct Args {
  int Q, H, n_kv, G, d_h, d_c, dcp, dhp;   // dcp, dhp: padded to whole 64-column boxes
  int gb, qb, n_gblk, n_qblk;              // KV heads and queries per unit, units per sequence
  int T_cap, NST;
  int skip_tile;                           // testing only: 1-based tile that is not copied (0 = none)
  float scale;                             // softmax scale x log2(e)
  MlaWindow win;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* seq_lens;
  const int32_t* rope_pair;
  const double* theta;
  mla_cache_t cache;
  int32_t* err;
  uint64_t wait_ns;
  uint32_t stage, off_qr, off_ring, off_xchg, off_bar;
};

enum { kBarFull = 0, kBarEmpty = 4, kBarQ = 8, kBarAccFull, kBarAccEmpty, kBarQlat, kBarS, kBarP = kBarS + 2,
       kBarO = kBarP + 2, kBarA = kBarO + 2, kBarDone, kBarX, kBarC = kBarX + 4, kBars = kBarC + 4 };

__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)r * 128u + (uint32_t)(((c ^ r) & 7) << 4); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// D[tmem] (+)= A[tmem] * B[smem]^T: A holds row r in lane r, two bf16 of K per 32-bit column.
__device__ __forceinline__ void mma_a_tmem(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc),
      "r"(accumulate)
      : "memory");
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}

// sum + the dot product of eight bf16 pairs.
__device__ __forceinline__ float dot8(uint4 u, uint4 v, float sum) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) sum = fmaf(hi_f(x[e]), hi_f(y[e]), fmaf(lo_f(x[e]), lo_f(y[e]), sum));
  return sum;
}

// Bits 0 .. n-1 of 64 (n outside [0, 64] cut to it).
__device__ __forceinline__ uint64_t below64(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// QB: code width of a quantised latent (4 or 2), 0 for bf16.
template <bool PAGED, int QB>
__global__ void __launch_bounds__(kThreadsOf<QB>, 1)
window_fused_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_kr,
                    const __grid_constant__ CUtensorMap tm_uk, const __grid_constant__ CUtensorMap tm_uv,
                    const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb - smem_u32(smem_raw));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto bar = [&](int i) { return sb + a.off_bar + 8u * (uint32_t)i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + a.off_bar + 8 * kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_tmem + 1);
  const uint64_t lim = a.wait_ns;
  const int NST = a.NST;

  // unit -> sequence, KV heads, queries
  const int u = blockIdx.x;
  const int qblk = u % a.n_qblk, gblk = (u / a.n_qblk) % a.n_gblk, b = u / (a.n_qblk * a.n_gblk);
  const int g0 = gblk * a.gb, ng = min(a.gb, a.n_kv - g0);
  const int q0 = qblk * a.qb, nq = min(a.qb, a.Q - q0);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < NST; ++s) { mbar_init(bar(kBarFull + s), 1); mbar_init(bar(kBarEmpty + s), 1); }
    const int rows[] = {kBarQ, kBarAccEmpty, kBarQlat, kBarP, kBarP + 1, kBarA};
    const int one[] = {kBarAccFull, kBarS, kBarS + 1, kBarO, kBarO + 1, kBarDone};
    for (int i : rows) mbar_init(bar(i), 8);   // the row warps
    for (int i : one) mbar_init(bar(i), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBarX + i), 2);   // the two warps of the same rows
    for (int i = 0; i < 4; ++i) mbar_init(bar(kBarC + i), 4);   // the dequantising warps
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int n_cbox = a.dcp / 64, n_hbox = a.dhp / 64;
  const uint32_t uk_bytes = (uint32_t)n_cbox * a.d_h * 128u, uv_bytes = (uint32_t)n_hbox * a.d_c * 128u;

  // The first W_uk slices belong to the plan: they may load before the kernels ahead are done.
  int loaded = 0;   // ring items issued (producer)
  auto load_uk = [&](int gi, int s) {
    mbar_expect_tx(bar(kBarFull + s), uk_bytes);
    for (int k = 0; k < n_cbox; ++k)
      tma_load_2d(sb + a.off_ring + (uint32_t)s * a.stage + k * a.d_h * 128, &tm_uk, bar(kBarFull + s), k * 64, (g0 + gi) * a.d_h);
    ++loaded;
  };
  if (warp == 0 && lane == 0)
    while (loaded < min(ng, NST)) load_uk(loaded, loaded);
  // rows (warps 4-11): thread -> row r of the unit, half hf of its tokens and columns
  const int w = warp & 3, hf = warp >= 8 && warp < 12, r = 32 * w + lane;   // tensor memory lane = row
  const int per_g = a.G * a.qb;
  const int gi = r / per_g, hi = (r / a.qb) % a.G, qi = r % a.qb;
  const bool valid = warp >= 4 && warp < 12 && gi < ng && qi < nq;
  const int g = g0 + gi;
  const size_t row = ((size_t)b * a.Q + q0 + qi) * a.H + g * a.G + hi;
  const uint32_t lane0 = tmem + ((uint32_t)(32 * w) << 16);
  float* xchg = reinterpret_cast<float*>(smem + a.off_xchg);   // [2][2 halves][rows]
  auto wwait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_spin(bar(i), parity, abort_flag, lim)); };
  int pair[2] = {0, 0};
  double theta[2] = {0, 0};
  if (valid) {
#pragma unroll
    for (int j = 0; j < 2; ++j) pair[j] = __ldg(a.rope_pair + g * 4 + 2 * hf + j);
#pragma unroll
    for (int j = 0; j < 2; ++j) theta[j] = __ldg(a.theta + pair[j]);
  }
  pdl_wait();   // queries, lengths and the cache come from earlier kernels
  pdl_trigger();

  // this thread's part of the q row: blocks hf, hf + 2, .. of 16 values, and two kept pairs
  uint4 qv[8];
  uint32_t xy[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = 2 * (hf + 2 * (j / 2)) + j % 2;
    qv[j] = valid && c < a.d_h / 8 ? __ldg(reinterpret_cast<const uint4*>(a.q + row * a.d_h) + c) : make_uint4(0, 0, 0, 0);
  }
  if (valid) {
#pragma unroll
    for (int j = 0; j < 2; ++j) xy[j] = __ldg(reinterpret_cast<const uint32_t*>(a.q + row * a.d_h) + pair[j]);
  }
  // what the unit reads
  int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > a.T_cap || (a.Q > 1 && L < a.Q)) {
    if (threadIdx.x == 0) raise_error(a.err, MLA_DEVERR_SEQ_LEN);
    L = 0;
  }
  const int p0 = L - a.Q + q0;                      // position of the unit's first query
  const Span span = L > 0 ? unit_span(p0 + nq, nq, kT, a.win) : Span();
  const int T = (span.len + kT - 1) / kT;           // tiles
  auto tile_token = [&](int n) { return span.token(n * kT); };

  if (warp < 4) {
    if (QB) setmaxnreg_dec<88>();
    if (warp == 0) {
      // ============================================================ TMA producer (lane 0)
      if (lane == 0) {
        const int items = T > 0 ? 2 * ng + T : 0;
        bool ok = true;
        RingPos rp;
        for (int i = 0; i < loaded; ++i) rp.next(NST);
        while (ok && loaded < items) {
          const int i = loaded, s = rp.slot;
          if (i >= NST) ok = mbar_spin(bar(kBarEmpty + s), rp.parity ^ 1, abort_flag, lim);
          if (!ok) break;
          rp.next(NST);
          if (i < ng) { load_uk(i, s); continue; }
          const uint32_t at = sb + a.off_ring + (uint32_t)s * a.stage;
          if (i < ng + T) {
            if (i - ng + 1 != a.skip_tile) {
              const int t = tile_token(i - ng);
              const MlaLoc lc = PAGED ? mla_loc(a.cache, b, t, a.err) : MlaLoc{b, t, a.T_cap};
              const int row = lc.pb * lc.cap + lc.pt;
              mbar_expect_tx(bar(kBarFull + s), (QB ? 0u : (uint32_t)n_cbox * kBox) + kKrTile);
              for (int k = 0; k < (QB ? 0 : n_cbox); ++k) tma_load_2d(at + k * kBox, &tm_c, bar(kBarFull + s), k * 64, row);
              tma_load_2d(at + n_cbox * kBox, &tm_kr, bar(kBarFull + s), g0 * 8, row);
            }
          } else {
            const int gi = i - ng - T;
            mbar_expect_tx(bar(kBarFull + s), uv_bytes);
            for (int k = 0; k < n_hbox; ++k)
              tma_load_2d(at + k * a.d_c * 128, &tm_uv, bar(kBarFull + s), k * 64, (g0 + gi) * a.d_c);
          }
          ++loaded;
        }
        volatile int never = 0;   // every copy lands before the CTA exits
        for (int i = max(0, loaded - NST); i < loaded; ++i) mbar_spin(bar(kBarFull + i % NST), (i / NST) & 1, &never, lim);
      }
    } else if (warp == 1) {
      // ============================================================ MMA issuer
      // The whole warp walks the same path, with every condition the same in all lanes, and one
      // elected lane issues: the compiler then keeps descriptors in uniform registers.  (Issued
      // from a branch of lane 0 a product took 110 to 190 cycles, more than most of them compute.)
      if (T > 0) {
        auto wait_all = [&](int i, int parity) {
          return __all_sync(0xffffffffu, mbar_spin(bar(i), parity, abort_flag, lim)) != 0;
        };
        auto ready = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_test(bar(i), parity)) != 0; };
        auto stage_at = [&](const RingPos& p) { return sb + a.off_ring + (uint32_t)p.slot * a.stage; };
        RingPos r1;   // ring items: weights, then tiles (S), then weights
        bool ok = wait_all(kBarQ, 0);
        // absorption: q (tensor memory) x W_ukF[g], once per KV head over all rows
        const uint32_t id_abs = idesc_bf16_f32(kRows, a.dcp, false, true);
        for (int gi = 0; ok && gi < ng; ++gi) {
          ok = wait_all(kBarFull + r1.slot, r1.parity) && (gi == 0 || wait_all(kBarAccEmpty, (gi - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t w0 = smem_desc(stage_at(r1), a.d_h * 128, 1024, kLayoutSW128);
            for (int k = 0; k < a.d_h / 16; ++k) mma_a_tmem(tmem + kOCol, tmem + kSCol + 8 * k, w0 + 128u * k, id_abs, k > 0);
            tc_commit(bar(kBarEmpty + r1.slot));
            tc_commit(bar(kBarAccFull));
          }
          __syncwarp();
          r1.next(NST);
        }
        ok = ok && wait_all(kBarQlat, 0);
        tc_fence_after();
        // tiles: S(n) needs its tile and the buffer of tile n - 2, whose P was read by O(n - 2)
        // issued before it; O(n) needs P(n).  Whichever can go next is issued.
        const uint32_t id_s = idesc_bf16_f32(kRows, kT, false, false), id_o = idesc_bf16_f32(kRows, a.dcp, false, true);
        // descriptors are made once; a step along K adds its bytes / 16 to the address field
        const uint64_t desc_q = smem_desc(sb, 16, 1024, kLayoutSW128), desc_qr = smem_desc(sb + a.off_qr, 16, 512, kLayoutSW64);
        int n1 = 0, n2 = 0;
        RingPos r2 = r1;     // tiles of O
        RingPos rc;          // dequantised tiles
        uint64_t idle = 0;   // when nothing could be issued: since when (read every 64th look only)
        int looks = 0;
        while (ok && n2 < T) {
          if (n1 < T && n1 <= n2 + 1 && ready(kBarFull + r1.slot, r1.parity) && (!QB || ready(kBarC + rc.slot, rc.parity))) {
            tc_fence_after();
            if (elect_one()) {
              const uint32_t c0 = stage_at(r1), d = tmem + kSCol + (n1 & 1) * kT;
              uint64_t da = desc_q, db = smem_desc(c0, 16, 1024, kLayoutSW128);
              const uint64_t dk = smem_desc(c0 + n_cbox * kBox, 16, 512, kLayoutSW64);
              tc_mma_bf16(d, desc_qr, dk, id_s, 0);
              if (ng > 2) tc_mma_bf16(d, desc_qr + 2, dk + 2, id_s, 1);
              for (int k = 0; k < n_cbox; ++k) {   // a box: four steps of 16 columns
                tc_mma_bf16(d, da, db, id_s, 1);
                tc_mma_bf16(d, da + 2, db + 2, id_s, 1);
                tc_mma_bf16(d, da + 4, db + 4, id_s, 1);
                tc_mma_bf16(d, da + 6, db + 6, id_s, 1);
                da += kBox >> 4;
                db += kBox >> 4;
              }
              tc_commit(bar(kBarS + (n1 & 1)));
            }
            __syncwarp();
            r1.next(NST);
            rc.next(NST);
            ++n1;
            looks = 0;
          } else if (n2 < n1 && ready(kBarP + (n2 & 1), (n2 >> 1) & 1)) {
            tc_fence_after();
            if (elect_one()) {
              const uint32_t p = tmem + kSCol + (n2 & 1) * kT;
              const uint64_t dv = smem_desc(stage_at(r2), kBox, 1024, kLayoutSW128);
              mma_a_tmem(tmem + kOCol, p, dv, id_o, n2 > 0);
  #pragma unroll
              for (int k = 1; k < kT / 16; ++k) mma_a_tmem(tmem + kOCol, p + 8 * k, dv + 128 * k, id_o, 1);
              tc_commit(bar(kBarEmpty + r2.slot));
              tc_commit(bar(kBarO + (n2 & 1)));
            }
            __syncwarp();
            r2.next(NST);
            ++n2;
            looks = 0;
          } else if ((++looks & 63) == 0) {
            const uint64_t now = globaltimer();
            if (looks == 64) idle = now;
            if (*abort_flag || now - idle > lim) { *abort_flag = 1; ok = false; }
            ok = __all_sync(0xffffffffu, ok) != 0;
          }
        }
        // output: merged latent (tensor memory, high and low halves) x W_uv[g]
        const uint32_t id_out = idesc_bf16_f32(kRows, a.dhp, false, true);
        ok = ok && wait_all(kBarA, 0);
        for (int gi = 0; ok && gi < ng; ++gi) {
          ok = wait_all(kBarFull + r1.slot, r1.parity) && (gi == 0 || wait_all(kBarAccEmpty, (ng + gi - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t w0 = smem_desc(stage_at(r1), a.d_c * 128, 1024, kLayoutSW128);
            for (int k = 0; k < a.d_c / 16; ++k) mma_a_tmem(tmem + kSCol + kT, tmem + kSCol + 8 * k, w0 + 128u * k, id_out, k > 0);
            for (int k = 0; k < a.d_c / 16; ++k) mma_a_tmem(tmem + kSCol + kT, tmem + kOCol + 8 * k, w0 + 128u * k, id_out, 1);
            tc_commit(bar(kBarEmpty + r1.slot));
            tc_commit(bar(kBarAccFull));
          }
          __syncwarp();
          r1.next(NST);
        }
        if (elect_one()) tc_commit(bar(kBarDone));   // whatever was issued has finished before tensor memory is freed
        __syncwarp();
        volatile int never = 0;
        mbar_spin(bar(kBarDone), 0, &never, lim);
      }
    }   // (warps 2 and 3 idle)
  } else if (QB != 0 && warp >= 12) {
    // ============================================================ dequantisation (a token row per thread)
    if (QB) setmaxnreg_dec<88>();
    constexpr int kQ = QB ? QB : 4;
    const int tr = 32 * w + lane, code_row = a.d_c * kQ / 8, groups = a.d_c / 32;
    // The codes come straight from the cache, a group of 32 ahead of the one in work (the first
    // touch of a row brings its whole line); where a tile's rows lie, their lines and group
    // scales are asked for a tile ahead.
    struct Src { long long row = -1; uint32_t sc[4] = {0, 0, 0, 0}; } cur, nxt;
    auto source = [&](int n, Src& o) {
      const int t0 = tile_token(n), t = t0 + tr;
      o.row = -1;
      // a row that no query of the unit sees is zero (its codes and scales may be stale)
      if (n >= T || tr >= span.len - n * kT || (t >= a.win.n_sink && t < span.lo)) return;
      const MlaLoc lc = PAGED ? mla_loc(a.cache, b, t0, a.err) : MlaLoc{b, t0, a.T_cap};
      o.row = (long long)lc.pb * lc.cap + lc.pt + tr;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(a.cache.c_kv) + o.row * code_row));
      const unsigned short* sp = reinterpret_cast<const unsigned short*>(a.cache.c_scales) + o.row * groups;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o.sc[k] = (2 * k < groups ? (uint32_t)__ldg(sp + 2 * k) : 0u) | (2 * k + 1 < groups ? (uint32_t)__ldg(sp + 2 * k + 1) << 16 : 0u);
    };
    if (T > 0) source(0, cur);
    bool ok = true;
    RingPos rt, rc;
    for (int i = 0; i < ng; ++i) rt.next(NST);
    for (int n = 0; ok && n < T; ++n, rt.next(NST), rc.next(NST)) {
      source(n + 1, nxt);
      const uint8_t* codes = reinterpret_cast<const uint8_t*>(a.cache.c_kv) + cur.row * code_row;
      auto group = [&](int g) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (cur.row < 0 || g >= groups) return v;
        if (kQ == 4) return __ldg(reinterpret_cast<const uint4*>(codes) + g);
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(codes) + g);
        return make_uint4(x.x, x.x >> 16, x.y, x.y >> 16);
      };
      uint4 ahead = group(0);
      if (n + ng >= NST) ok = wwait(kBarEmpty + rt.slot, rt.parity ^ 1);
      if (!ok) break;
      uint8_t* C = smem + a.off_ring + (uint32_t)rt.slot * a.stage;
      auto put = [&](int chunk, uint4 v) { *reinterpret_cast<uint4*>(C + (chunk >> 3) * kBox + sw128(tr, chunk)) = v; };
      // (rolled loops: little code, for the instruction caches)
#pragma unroll 1
      for (int g = 0; g < groups; ++g) {
        uint4 wd = ahead;
        ahead = group(g + 1);
        const float sv = __half2float(__ushort_as_half((unsigned short)cur.sc[0]));
#pragma unroll
        for (int k = 0; k < 4; ++k) cur.sc[k] = __funnelshift_r(cur.sc[k], k < 3 ? cur.sc[k + 1] : 0u, 16);   // the next group's scale
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          put(4 * g + ch, cur.row >= 0 ? dequant8<kQ>(wd.x, sv) : make_uint4(0, 0, 0, 0));
          wd.x = wd.y; wd.y = wd.z; wd.z = wd.w;
        }
      }
      for (int c = a.d_c / 8; c < a.dcp / 8; ++c) put(c, make_uint4(0, 0, 0, 0));   // padding columns
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarC + rc.slot));
      cur = nxt;
    }
  } else {
    // ============================================================ rows
    if (QB) setmaxnreg_inc<168>();
    // Two threads per row, in warps w and w + 4 of the same tensor memory lanes: each takes
    // half of every tile's tokens and of every accumulator's columns.
    auto arrive = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    int n_sync = 0;
    auto pair_sync = [&]() {   // with the other warp of these rows (bounded, unlike a named barrier)
      tc_fence_before();
      arrive(kBarX + w);
      const bool met = wwait(kBarX + w, n_sync++ & 1);
      tc_fence_after();
      return met;
    };
    if (T == 0) {   // an empty sequence: zero rows
      if (valid)
        for (int c = hf; c < a.d_h / 8; c += 2) reinterpret_cast<uint4*>(a.out + row * a.d_h)[c] = make_uint4(0, 0, 0, 0);
    } else {
      // q row into tensor memory (blocks of 16 values in turn), the rotated kept pairs, scaled,
      // into this row's KV head chunk of the block-diagonal RoPE operand
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (8 * (hf + 2 * j) < a.d_h / 2) {
          const uint32_t v[8] = {qv[2 * j].x, qv[2 * j].y, qv[2 * j].z, qv[2 * j].w,
                                 qv[2 * j + 1].x, qv[2 * j + 1].y, qv[2 * j + 1].z, qv[2 * j + 1].w};
          tmem_st8(lane0 + kSCol + 8 * (hf + 2 * j), v);
        }
      }
      {
        uint32_t rot[2] = {0, 0};
        if (valid) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // the special-function unit's sine and cosine of an angle reduced to [-pi, pi]:
            // about 5e-7 off, against the 2^-8 of the bf16 rounding that follows
            float sn, cs;
            __sincosf(rope_angle(p0 + qi, theta[j]), &sn, &cs);
            const float x = lo_f(xy[j]), y = hi_f(xy[j]);
            rot[j] = pack2((x * cs - y * sn) * a.scale, (x * sn + y * cs) * a.scale);
          }
        }
        uint8_t* qr = smem + a.off_qr + r * 64;
#pragma unroll
        for (int c = 0; c < kMaxG; ++c)
          *reinterpret_cast<uint2*>(qr + ((c ^ (r >> 1)) & 3) * 16 + 8 * hf) = c == gi ? make_uint2(rot[0], rot[1]) : make_uint2(0, 0);
      }
      tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(kBarQ);
      // Q_lat: the accumulator's rows of each KV head, scaled, rounded once to bf16 (the type of the
      // latents that it meets in S), which makes 0.0016 of the output's norm; in two halves it would
      // take twice its shared memory and S's products
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok && k < ng; ++k) {
        ok = wwait(kBarAccFull, k & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = hf * (a.dcp / 2); c0 < (hf + 1) * (a.dcp / 2); c0 += 32) {
          uint32_t v[32];
          tmem_ld32(lane0 + kOCol + c0, v);
          tmem_wait_ld();
          if (gi != k && !(gi >= ng && k == 0)) continue;   // rows of no KV head: once, whatever they hold
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack2(__uint_as_float(v[8 * j + 2 * e]) * a.scale, __uint_as_float(v[8 * j + 2 * e + 1]) * a.scale);
            const int ch = c0 / 8 + j;
            *reinterpret_cast<uint4*>(smem + (ch >> 3) * kBox + sw128(r, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc_fence_before();
        arrive(kBarAccEmpty);
      }
      fence_proxy_async_smem();
      if (ok) arrive(kBarQlat);
      // tiles: this thread's tokens are [64 hf, 64 hf + 64) of each
      const int p_row = valid ? p0 + qi : -1;
      float m = -INFINITY, l = 0.f;
      RingPos rt;
      for (int i = 0; i < ng; ++i) rt.next(NST);
#pragma unroll 1
      for (int n = 0; ok && n < T; ++n, rt.next(NST)) {
        const int t0 = tile_token(n), nvalid = min(kT, span.len - n * kT);
        ok = wwait(kBarS + (n & 1), (n >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t scol = lane0 + kSCol + (n & 1) * kT;
        float s[64];
        {
          uint32_t raw[2][32];
          tmem_ld32(scol + 64 * hf, raw[0]);
          tmem_ld32(scol + 64 * hf + 32, raw[1]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            asm volatile("" : "+r"(raw[e / 32][e % 32]));   // the values exist only after the wait
            s[e] = __uint_as_float(raw[e / 32][e % 32]);
          }
        }
        // tiles whose tokens every query of the unit sees need no mask
        const bool whole = nvalid == kT && t0 + kT - 1 <= p0 && (t0 > p0 + nq - 1 - a.win.window || t0 + kT <= a.win.n_sink);
        if (!whole) {
          const int h0 = t0 + 64 * hf;
          const int lim_t = min(nvalid - 64 * hf, p_row + 1 - h0);
          const int sink_t = a.win.n_sink - h0, win_t = p_row + 1 - a.win.window - h0;
          // bit t: token t of the half is before lim_t, and before sink_t or from win_t on
          const uint64_t seen = below64(lim_t) & (below64(sink_t) | ~below64(win_t));
#pragma unroll
          for (int t = 0; t < 64; ++t) s[t] = ((uint32_t)(seen >> (t & 32)) >> (t & 31)) & 1u ? s[t] : -INFINITY;
          // rows that no query of the unit sees (stale or hidden, possibly not finite) are
          // zeroed before O's product multiplies them by P = 0; S of this tile has been read
          if (!QB) {
            uint8_t* C = smem + a.off_ring + (uint32_t)rt.slot * a.stage;
            auto zero_rows = [&](int from, int to) {   // consecutive threads, consecutive 16-byte chunks
              for (int i = from * 8 + 128 * hf + r; i < to * 8; i += 256)
                for (int k = 0; k < n_cbox; ++k) *reinterpret_cast<uint4*>(C + k * kBox + i * 16) = make_uint4(0, 0, 0, 0);
            };
            zero_rows(max(0, a.win.n_sink - t0), min(nvalid, span.lo - t0));
            zero_rows(nvalid, kT);
            fence_proxy_async_smem();
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 64; ++t) mx[t & 3] = max_nan(mx[t & 3], s[t]);
        float mine = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
        if (mine != mine && valid) {
          // A key that is not finite: the other KV heads' zeros times it are NaN.  The scores that
          // came out NaN once more, with the row's own key (a latent that is not finite makes them
          // NaN by the definition too); the tile stays until P is written.  (The test costs the
          // Llama-shaped chunk 0.6 us of 34, the narrow one 0.3 of 17.)
          uint64_t bad = 0;
#pragma unroll
          for (int t = 0; t < 64; ++t) bad |= s[t] != s[t] ? 1ull << t : 0ull;
          (void)mbar_spin(bar(kBarFull + rt.slot), rt.parity, abort_flag, lim);   // (complete: S is)
          if (QB) (void)mbar_spin(bar(kBarC + n % NST), (n / NST) & 1, abort_flag, lim);
          const uint8_t* C = smem + a.off_ring + (uint32_t)rt.slot * a.stage;
          const uint8_t* K = C + n_cbox * kBox;
          const uint4 qr = *reinterpret_cast<const uint4*>(smem + a.off_qr + r * 64 + ((gi ^ (r >> 1)) & 3) * 16);
#pragma unroll 1
          while (bad) {
            const int t = __ffsll(bad) - 1, tt = 64 * hf + t;
            bad &= bad - 1;
            float v = 0.f, zero = 0.f;   // zero: stays 0 while the latent is finite
#pragma unroll 1
            for (int c = 0; zero == 0.f && c < a.d_c / 8; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(C + (c >> 3) * kBox + sw128(tt, c));
              zero = dot8(x, make_uint4(0, 0, 0, 0), zero);
              v = dot8(x, *reinterpret_cast<const uint4*>(smem + (c >> 3) * kBox + sw128(r, c)), v);
            }
            v = dot8(*reinterpret_cast<const uint4*>(K + tt * 64 + ((gi ^ (tt >> 1)) & 3) * 16), qr, v + zero);
#pragma unroll
            for (int k = 0; k < 64; ++k) s[k] = k == t ? v : s[k];
          }
          mine = -INFINITY;
#pragma unroll
          for (int t = 0; t < 64; ++t) mine = fmaxf(mine, s[t]);
        }
        // the row's maximum over both halves; past this barrier both have read their S, so P
        // may go over it
        float* xm = xchg + (n & 1) * 2 * kRows;
        xm[hf * kRows + r] = mine;
        ok = pair_sync();
        if (!ok) break;
        const float top = fmaxf(xm[r], xm[kRows + r]);
        // The running max is raised when a row outgrew it by more than kTau (P stays below
        // 2^kTau, in range for bf16 and the float32 sums); the loads and stores of O are
        // warp-collective, so the other rows multiply by 1.
        const bool raise = top > m + kTau;
        if (__any_sync(0xffffffffu, raise)) {
          const float al = raise ? exp2f(m - top) : 1.f;   // m = -inf: 0
          if (n > 0) {
            ok = wwait(kBarO + ((n - 1) & 1), ((n - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = hf * (a.dcp / 2); c0 < (hf + 1) * (a.dcp / 2); c0 += 32) {
              uint32_t o[32];
              tmem_ld32(lane0 + kOCol + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
              tmem_st32(lane0 + kOCol + c0, o);
            }
          }
          if (raise) {
            l *= al;
            m = top;
          }
        }
        const float mb = m == -INFINITY ? 0.f : m;   // masked scores are -inf: 2^(-inf) = 0
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // P, rounded to bf16: both operands of a product have the latent's type.  Tokens' errors are
        // independent: 0.0012 of the output's norm over few visible tokens, less over many, where the
        // output's own rounding makes 0.0017; P in two halves would double O's products, which bound
        // the kernel while tiles flow.
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = ex2_approx(s[2 * e] - mb), y = ex2_approx(s[2 * e + 1] - mb);
          sum[(2 * e) & 3] += x;
          sum[(2 * e + 1) & 3] += y;
          pk[e] = pack2(x, y);
        }
        tmem_st32(scol + 32 * hf, pk);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        arrive(kBarP + (n & 1));
      }
      // merged latent, normalised, in two bf16 halves (so that this rounding does not count):
      // the high ones over S, the low ones, once both threads have read their part, over O
      if (ok) ok = wwait(kBarO + ((T - 1) & 1), ((T - 1) >> 1) & 1);
      if (ok) {
        float* xl = xchg + (T & 1) * 2 * kRows;   // (the last tile's maxima may still be read)
        xl[hf * kRows + r] = l;
        ok = pair_sync();
        const float den = xl[r] + xl[kRows + r];
        const float inv = 1.f / den;   // (every score -inf: 0 / 0, as the definition has it)
        const int half = a.d_c / 2, c_at = hf * half;   // a multiple of 16 up to 128
        uint32_t lo2[8][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (16 * j >= half) continue;
          uint32_t v[16], hi2[8];
          tmem_ld16(lane0 + kOCol + c_at + 16 * j, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            asm volatile("" : "+r"(v[2 * e]), "+r"(v[2 * e + 1]));
            const float x = __uint_as_float(v[2 * e]) * inv, y = __uint_as_float(v[2 * e + 1]) * inv;
            hi2[e] = pack2(x, y);
            lo2[j][e] = pack2(x - lo_f(hi2[e]), y - hi_f(hi2[e]));
          }
          tmem_st8(lane0 + kSCol + c_at / 2 + 8 * j, hi2);
        }
        ok = pair_sync() && ok;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (16 * j < half) tmem_st8(lane0 + kOCol + c_at / 2 + 8 * j, lo2[j]);
        tmem_wait_st();
        tc_fence_before();
        arrive(kBarA);
      }
#pragma unroll 1
      for (int k = 0; ok && k < ng; ++k) {
        ok = wwait(kBarAccFull, (ng + k) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 16 * hf; c0 < a.d_h; c0 += 32) {
          uint32_t v[16];
          tmem_ld16(lane0 + kSCol + kT + c0, v);
          tmem_wait_ld();
          if (!valid || gi != k) continue;
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * a.d_h + c0);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack2(__uint_as_float(v[8 * j + 2 * e]), __uint_as_float(v[8 * j + 2 * e + 1]));
            dst[j] = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc_fence_before();
        arrive(kBarAccEmpty);
      }
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

static bool map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t gdim[2] = {cols, rows};
  cuuint64_t gstride[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout {
  int NST;
  uint32_t stage, off_qr, off_ring, off_xchg, off_bar, total;
};
// [Q_lat boxes][RoPE queries][ring of 2 to 4 stages][row exchange][barriers]
static Layout layout(int dcp) {
  Layout L{};
  const uint32_t n_cbox = dcp / 64;
  L.stage = n_cbox * kBox + kKrTile;
  L.off_qr = n_cbox * kBox;
  L.off_ring = L.off_qr + kRows * 64;
  const uint32_t tail = 4 * kRows * 4 + 8 * kBars + 16;
  L.NST = (int)std::min<uint32_t>(4, (kSmemMax - 1024 - L.off_ring - tail) / L.stage);
  L.off_xchg = L.off_ring + L.NST * L.stage;
  L.off_bar = L.off_xchg + 4 * kRows * 4;
  L.total = L.off_xchg + tail + 1024;
  return L;
}

// KV heads per unit: few of them re-read the window more often but fill the machine and its
// rows' products; the candidate with the least (rounds of CTAs) x (time of a unit) is taken.
// Times in units of a tile's products at d_c = 256: a tile 1, a unit's ends 2, a KV head's weights 2.
static int pick_gb(int B, int Q, int G, int n_kv, int tiles, int sms) {
  int best = 1;
  double best_cost = 1e30;
  for (int gb = 1; gb <= kMaxG && gb <= n_kv && gb * G <= kRows; gb *= 2) {
    const int qb = std::min(Q, kRows / (gb * G));
    const long long units = (long long)B * ((n_kv + gb - 1) / gb) * ((Q + qb - 1) / qb);
    const double cost = (double)((units + sms - 1) / sms) * (tiles + 2.0 + 2.0 * gb);
    if (cost < best_cost) { best_cost = cost; best = gb; }
  }
  return best;
}

}  // namespace fused
}  // namespace mla

// Shapes: bf16 weights, latent in bf16 or 4- or 2-bit groups, r = 4 kept pairs, d_c a multiple of 32 up to 256, head dim a
// multiple of 16 up to 128, at most 128 query heads per KV head, RoPE rows of whole 16 bytes.
bool mla_window_fused_capable(const mla_plan& p) {
  const mla_config_t& c = p.cfg;
  return c.dtype == MLA_BF16 && c.cache_kind != MLA_CACHE_INT4_G32_R128 && c.r_pairs == 4 && c.d_c % 32 == 0 && c.d_c <= 256 &&
         c.head_dim % 16 == 0 && c.head_dim <= 128 && c.n_heads / c.n_kv_heads <= 128;
}

cudaError_t mla_launch_window_fused(const mla_plan& p, const mla_cache_t& c, const int32_t* seq_lens, const void* q,
                                    int B, int Q, void* out, MlaWindow win, cudaStream_t s) {
  using namespace mla::fused;
  const mla_config_t& cfg = p.cfg;
  Args a;
  a.Q = Q; a.H = cfg.n_heads; a.n_kv = cfg.n_kv_heads; a.G = a.H / a.n_kv; a.d_h = cfg.head_dim; a.d_c = cfg.d_c;
  a.dcp = (a.d_c + 63) / 64 * 64; a.dhp = (a.d_h + 63) / 64 * 64;
  const int tiles = (int)std::min<long long>((long long)c.T_cap, (long long)win.n_sink + win.window + Q) / kT + 1;
  a.gb = pick_gb(B, Q, a.G, a.n_kv, tiles, p.num_sms);
  a.qb = std::min(Q, kRows / (a.gb * a.G));
  a.n_gblk = (a.n_kv + a.gb - 1) / a.gb;
  a.n_qblk = (Q + a.qb - 1) / a.qb;
  const long long units = (long long)B * a.n_gblk * a.n_qblk;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  a.T_cap = c.T_cap; a.skip_tile = p.opt_skip_tile;
  a.scale = mla::kLog2e * (cfg.softmax_scale > 0.0f ? cfg.softmax_scale : (float)(1.0 / sqrt((double)cfg.head_dim)));
  a.win = win;
  a.q = (const __nv_bfloat16*)q; a.out = (__nv_bfloat16*)out; a.seq_lens = seq_lens;
  a.rope_pair = p.rope_pair; a.theta = p.theta; a.cache = c; a.err = p.err;
  a.wait_ns = (uint64_t)p.opt_wait_us * 1000u;
  const Layout L = layout(a.dcp);
  a.NST = L.NST; a.stage = L.stage; a.off_qr = L.off_qr; a.off_ring = L.off_ring; a.off_xchg = L.off_xchg; a.off_bar = L.off_bar;
  const uint64_t rows = mla_cache_rows(c);
  CUtensorMap tm_c, tm_kr, tm_uk, tm_uv;
  const int qbits = mla_kind_quant(cfg.cache_kind) ? mla_quant_bits(cfg.cache_kind) : 0;   // (no map of codes)
  if (!map_2d(&tm_c, qbits ? p.W_ukF : c.c_kv, a.d_c, qbits ? (uint64_t)a.d_h : rows, 64, qbits ? a.d_h : kT) || !map_2d(&tm_kr, c.k_rope, p.R, rows, 32, kT) ||
      !map_2d(&tm_uk, p.W_ukF, a.d_c, (uint64_t)a.n_kv * a.d_h, 64, a.d_h) ||
      !map_2d(&tm_uv, p.W_uv, a.d_h, (uint64_t)a.n_kv * a.d_c, 64, a.d_c))
    return cudaErrorInvalidValue;
  auto pick = [&](auto paged) {
    constexpr bool PAGED = decltype(paged)::value;
    return qbits == 4 ? window_fused_kernel<PAGED, 4> : qbits == 2 ? window_fused_kernel<PAGED, 2> : window_fused_kernel<PAGED, 0>;
  };
  const auto kern = c.block_table ? pick(std::true_type()) : pick(std::false_type());
  cudaError_t e = mla_smem_limit(p, (const void*)kern, L.total);
  if (e != cudaSuccess) return e;
  if ((e = mla_profile_event(p, kProfAttention, false, s)) != cudaSuccess) return e;
  e = mla_launch_kernel(kern, dim3((unsigned)units), dim3(qbits ? kThreadsOf<4> : kThreadsOf<0>), L.total, s, p.opt_pdl, tm_c, tm_kr, tm_uk, tm_uv, a);
  if (e != cudaSuccess) return e;
  return mla_profile_event(p, kProfAttention, true, s);
}
