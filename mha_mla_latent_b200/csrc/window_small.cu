// Windowed decode of small problems in one launch: a CTA takes one sequence and one KV head's
// query heads from the raw queries to the finished output, on the CUDA cores in float32.
//
// Paper notes "MHA2MLA" (ACL 2025), §关键设计: the absorbed query scores against the latent, the
// partial-RoPE term is added, the weighted latent goes through W_uv.  With few visible tokens
// the three launches of the split form (absorption, attention, merge) and their waits cost more
// than the work; here nothing passes through memory between the steps.  Every KV head reads the
// sequence's latents again (from the L2), which is what limits the size it is taken for.
//
// The CTA's slices of W_uk and W_uv belong to the plan: they are copied to shared memory before
// the kernel ahead is waited for.  Only visible tokens are read.  Scores, probabilities and sums
// are float32; nothing is rounded before the output.
#include <algorithm>

#include "decode_common.cuh"
#include "sm100.cuh"

namespace mla {
namespace wsmall {

using namespace sm100;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTokens = 1024 + 128;   // visible tokens: scores in shared memory

struct Args {
  int H, n_kv, d_h, r, d_c, T_cap;
  float scale;                // softmax scale x log2(e)
  MlaWindow win;
  const void* q;              // [B][H][d_h]
  const void* W_ukF;          // [n_kv][d_h][d_c]
  const void* W_uv;           // [n_kv][d_c][d_h]
  const int32_t* rope_pair;
  const double* theta;
  const int32_t* seq_lens;
  void* out;
  mla_cache_t cache;
  int32_t* err;
  uint32_t off_uv, off_q, off_lat, off_rope, off_p, off_part;   // shared memory, bytes
};

// 16 bytes of T as float.
__device__ __forceinline__ void unpack(uint4 v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// G: query heads of a KV head.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) window_small_kernel(const __grid_constant__ Args a) {
  constexpr int V = 16 / sizeof(T);   // values per 16-byte load
  extern __shared__ __align__(16) uint8_t smem[];
  T* s_uk = reinterpret_cast<T*>(smem);                             // [d_h][d_c]
  T* s_uv = reinterpret_cast<T*>(smem + a.off_uv);                  // [d_c][d_h]
  float* s_q = reinterpret_cast<float*>(smem + a.off_q);            // [G][d_h]
  float* s_lat = reinterpret_cast<float*>(smem + a.off_lat);        // [G][d_c]: absorbed query, then merged latent
  float* s_rope = reinterpret_cast<float*>(smem + a.off_rope);      // [G][2r]
  float* s_p = reinterpret_cast<float*>(smem + a.off_p);            // [G][kMaxTokens]
  float* s_part = reinterpret_cast<float*>(smem + a.off_part);      // [kThreads][G][V] partial sums
  __shared__ float s_inv[G];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.n_kv, g = blockIdx.x % a.n_kv;
  const int dh = a.d_h, dc = a.d_c, r2 = 2 * a.r;
  {
    const int n = dh * dc / V;   // whole 16-byte units: d_c is a multiple of V
    const T* uk = (const T*)a.W_ukF + (size_t)g * dh * dc;
    const T* uv = (const T*)a.W_uv + (size_t)g * dh * dc;
    for (int i = tid; i < n; i += kThreads) cp_async16(smem_u32(s_uk + i * V), uk + (size_t)i * V, 16);
    cp_async_commit();
    for (int i = tid; i < n; i += kThreads) cp_async16(smem_u32(s_uv + i * V), uv + (size_t)i * V, 16);
    cp_async_commit();
  }
  // the kept pair of this thread (head, pair), for the first G * r threads
  const bool rot = tid < G * a.r;
  const int pair = rot ? __ldg(a.rope_pair + g * a.r + tid % a.r) : 0;
  const double th = rot ? __ldg(a.theta + pair) : 0.0;
  pdl_wait();
  pdl_trigger();
  const size_t row0 = (size_t)b * a.H + (size_t)g * G;
  const T* q = (const T*)a.q + row0 * dh;
  for (int i = tid; i < G * dh; i += kThreads) s_q[i] = to_f32(q[i]);
  int L = __ldg(a.seq_lens + b);
  if (L < 0 || L > a.T_cap) {
    if (tid == 0) raise_error(a.err, MLA_DEVERR_SEQ_LEN);
    L = 0;
  }
  // visible tokens: the sinks ahead of the window, then the window
  const int lo = max(0, L - a.win.window), ns = min(a.win.n_sink, lo), n = ns + L - lo;
  auto token = [&](int i) { return i < ns ? i : lo + i - ns; };
  auto row_of = [&](int t) {
    const MlaLoc lc = mla_loc(a.cache, b, t, a.err);
    return (size_t)lc.pb * lc.cap + lc.pt;
  };
  asm volatile("cp.async.wait_group 1;" ::: "memory");   // W_uk
  __syncthreads();
  // 1. absorbed query: thread (column, part of the head dims); rotated kept pairs
  {
    const int parts = max(1, kThreads / dc), per = (dh + parts - 1) / parts;
    for (int c0 = 0; c0 < dc; c0 += kThreads) {
      const int c = c0 + tid % (parts > 1 ? dc : kThreads), part = parts > 1 ? tid / dc : 0;
      float acc[G] = {};
      if (c < dc && part < parts) {
        for (int d = part * per; d < min(dh, (part + 1) * per); ++d) {
          const float w = to_f32(s_uk[d * dc + c]);
#pragma unroll
          for (int h = 0; h < G; ++h) acc[h] += s_q[h * dh + d] * w;
        }
#pragma unroll
        for (int h = 0; h < G; ++h) s_part[(part * G + h) * dc + c] = acc[h];   // parts * dc <= kThreads, or one part
      }
    }
    if (rot) {
      const int h = tid / a.r, j = tid % a.r;
      const double x0 = s_q[h * dh + 2 * pair], x1 = s_q[h * dh + 2 * pair + 1];
      float sn, cs;
      rope_sincos(max(L - 1, 0), th, &sn, &cs);
      s_rope[h * r2 + 2 * j] = (float)((x0 * cs - x1 * sn) * (double)a.scale);
      s_rope[h * r2 + 2 * j + 1] = (float)((x0 * sn + x1 * cs) * (double)a.scale);
    }
    __syncthreads();
    for (int i = tid; i < G * dc; i += kThreads) {
      const int h = i / dc, c = i % dc;
      float s = 0.f;
      for (int k = 0; k < parts; ++k) s += s_part[(k * G + h) * dc + c];
      s_lat[i] = s * a.scale;
    }
    __syncthreads();
  }
  // 2. scores: LPT lanes per token, each on 16-byte units LPT apart of its row
  const int units = dc / V;
  {
    int LPT = 1;
    while (LPT < units && LPT < 32) LPT <<= 1;
    const int sub = lane & (LPT - 1), tpw = 32 / LPT;   // tokens per warp and step
    const T* c_kv = (const T*)a.cache.c_kv;
    const T* k_rope = (const T*)a.cache.k_rope;
    constexpr int kFly = 4;   // tokens in flight per lane: loads are unconditional, past the end on the last token
    // this lane's part of the queries: its first unit of the row, zeros past the row's end
    float ql[G][V], qr[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
      for (int e = 0; e < V; ++e) ql[h][e] = sub < units ? s_lat[h * dc + sub * V + e] : 0.f;
      qr[h] = sub < r2 ? s_rope[h * r2 + sub] : 0.f;
    }
    for (int i0 = warp * tpw; i0 < n; i0 += kFly * kWarps * tpw) {
      size_t row[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k) row[k] = row_of(token(min(i0 + k * kWarps * tpw + lane / LPT, n - 1)));
      uint4 v[kFly];
      float x[kFly];
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        v[k] = __ldg(reinterpret_cast<const uint4*>(c_kv + row[k] * dc) + min(sub, units - 1));
        x[k] = r2 > 0 ? to_f32(__ldg(k_rope + (row[k] * a.n_kv + g) * r2 + min(sub, r2 - 1))) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < kFly; ++k) {
        if (i0 + k * kWarps * tpw >= n) break;   // (the whole warp)
        float acc[G] = {}, c0[V];
        unpack(v[k], c0);
        if (sub < units) {   // (a lane past the row's end holds another unit, which may not be finite)
#pragma unroll
          for (int h = 0; h < G; ++h) {
#pragma unroll
            for (int e = 0; e < V; ++e) acc[h] += ql[h][e] * c0[e];
          }
        }
        for (int u = sub + LPT; u < units; u += LPT) {   // rows of more than 512 bytes
          float c[V];
          unpack(__ldg(reinterpret_cast<const uint4*>(c_kv + row[k] * dc) + u), c);
#pragma unroll
          for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < V; ++e) acc[h] += s_lat[h * dc + u * V + e] * c[e];
        }
        if (sub < r2) {
#pragma unroll
          for (int h = 0; h < G; ++h) acc[h] += qr[h] * x[k];
        }
        for (int j = sub + LPT; j < r2; j += LPT) {
          const float y = to_f32(__ldg(k_rope + (row[k] * a.n_kv + g) * r2 + j));
#pragma unroll
          for (int h = 0; h < G; ++h) acc[h] += s_rope[h * r2 + j] * y;
        }
        const int i = i0 + k * kWarps * tpw + lane / LPT;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          for (int o = LPT >> 1; o > 0; o >>= 1) acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], o);
          if (sub == 0 && i < n) s_p[h * kMaxTokens + i] = acc[h];
        }
      }
    }
    __syncthreads();
  }
  // 3. softmax, a warp per head
  if (warp < G) {
    float* p = s_p + warp * kMaxTokens;
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, p[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int i = lane; i < n; i += 32) {
      const float e = exp2f(p[i] - m);
      p[i] = e;
      l += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) s_inv[warp] = n > 0 ? 1.f / l : 0.f;
  }
  __syncthreads();
  // 4. weighted latent: thread (16-byte unit of the row, group of tokens)
  {
    const int groups = max(1, kThreads / units);
    for (int u0 = 0; u0 < units; u0 += kThreads) {
      const int u = u0 + (groups > 1 ? tid % units : tid), grp = groups > 1 ? tid / units : 0;
      float acc[G][V] = {};
      if (u < units && grp < groups) {
        constexpr int kFly = 8;   // rows in flight: past the end the last row again
        for (int i0 = grp; i0 < n; i0 += kFly * groups) {
          uint4 v[kFly];
#pragma unroll
          for (int k = 0; k < kFly; ++k)
            v[k] = __ldg(reinterpret_cast<const uint4*>((const T*)a.cache.c_kv + row_of(token(min(i0 + k * groups, n - 1))) * dc) + u);
#pragma unroll
          for (int k = 0; k < kFly; ++k) {
            const int i = i0 + k * groups;
            if (i >= n) break;
            float c[V];
            unpack(v[k], c);
#pragma unroll
            for (int h = 0; h < G; ++h) {
              const float p = s_p[h * kMaxTokens + i];
#pragma unroll
              for (int e = 0; e < V; ++e) acc[h][e] += p * c[e];
            }
          }
        }
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
          for (int e = 0; e < V; ++e) s_part[(grp * G + h) * dc + u * V + e] = acc[h][e];
      }
    }
    cp_async_wait_all();   // W_uv
    __syncthreads();
    for (int i = tid; i < G * dc; i += kThreads) {
      const int h = i / dc, c = i % dc;
      float s = 0.f;
      for (int k = 0; k < groups; ++k) s += s_part[(k * G + h) * dc + c];
      s_lat[i] = s * s_inv[h];
    }
    __syncthreads();
  }
  // 5. output: thread (head dim, part of the latent columns)
  {
    const int parts = max(1, kThreads / dh), per = (dc + parts - 1) / parts;
    for (int d0 = 0; d0 < dh; d0 += kThreads) {
      const int d = d0 + tid % (parts > 1 ? dh : kThreads), part = parts > 1 ? tid / dh : 0;
      if (d < dh && part < parts) {
        float acc[G] = {};
        for (int c = part * per; c < min(dc, (part + 1) * per); ++c) {
          const float w = to_f32(s_uv[c * dh + d]);
#pragma unroll
          for (int h = 0; h < G; ++h) acc[h] += s_lat[h * dc + c] * w;
        }
#pragma unroll
        for (int h = 0; h < G; ++h) s_part[(part * G + h) * dh + d] = acc[h];
      }
    }
    __syncthreads();
    for (int i = tid; i < G * dh; i += kThreads) {
      const int h = i / dh, d = i % dh;
      float s = 0.f;
      for (int k = 0; k < parts; ++k) s += s_part[(k * G + h) * dh + d];
      ((T*)a.out)[(row0 + h) * dh + d] = from_f32<T>(s);
    }
  }
}

struct Layout {
  uint32_t off_uv, off_q, off_lat, off_rope, off_p, off_part, total;
};
static Layout layout(const mla_config_t& c) {
  const int G = c.n_heads / c.n_kv_heads, eb = c.dtype == MLA_F32 ? 4 : 2, V = 16 / eb;
  auto up = [](size_t x) { return (x + 15) & ~(size_t)15; };
  Layout L;
  size_t o = up((size_t)c.head_dim * c.d_c * eb);
  L.off_uv = (uint32_t)o; o += up((size_t)c.head_dim * c.d_c * eb);
  L.off_q = (uint32_t)o; o += up((size_t)G * c.head_dim * 4);
  L.off_lat = (uint32_t)o; o += up((size_t)G * c.d_c * 4);
  L.off_rope = (uint32_t)o; o += up((size_t)G * 2 * c.r_pairs * 4 + 4);
  L.off_p = (uint32_t)o; o += up((size_t)G * kMaxTokens * 4);
  // partial sums: a slot per thread, head and value; at least one row of each kind
  const size_t part = std::max<size_t>((size_t)kThreads * V, std::max(c.head_dim, c.d_c));
  L.off_part = (uint32_t)o; o += up((size_t)G * part * 4);
  L.total = (uint32_t)o;
  return L;
}

}  // namespace wsmall
}  // namespace mla

// Shapes: up to 4 query heads per KV head, an unquantised cache of whole 16-byte rows.
static bool small_shape(const mla_plan& p) {
  const mla_config_t& c = p.cfg;
  const int G = c.n_heads / c.n_kv_heads, eb = c.dtype == MLA_F32 ? 4 : 2;
  return c.cache_kind == MLA_CACHE_SAME && G <= 4 && c.d_c * eb % 16 == 0 && c.head_dim * c.d_c * eb % 16 == 0 &&
         G * c.r_pairs <= mla::wsmall::kThreads && mla::wsmall::layout(c).total <= 200 * 1024;
}

// The rule, from device times of 16 layers (1 to 32 KV heads, 1 to 4 query heads each, d_c 32 to
// 256) at 1 to 192 sequences and 16 to 1100 visible tokens, one launch against the others:
// where those run on the CUDA cores (float32, other numbers of kept pairs) it is always the faster
// one (9 heads, r = 3, 16 sequences: 7.0 / 20.9 us at 16 tokens, 19.5 / 34.4 at 1100; float32, 32
// heads, d_c = 128, 192 sequences: 124 / 333 and 1373 / 4231).  The tensor-core launches take 10
// to 15 us (up to 32 heads) or 18 to 23 (the head-row kernel, more heads) while the call is small,
// which is met by an estimate of this kernel: a CTA takes 6 us, time for its weights, and per token
// the lanes of a row (a power of two of 16-byte units) times 1.6 ns + 0.5 per query head, a quarter
// more with two CTAs on an SM; with more CTAs than run at once it is behind.  Crossings: 32 heads
// over 32 KV heads, 4 sequences, d_c = 64 13.0 / 13.0 us at 400 tokens, d_c = 256 12.6 / 15.0 at 64
// and 17.0 / 15.4 at 128; 9 heads over 3, d_c = 32, 16 sequences 11.1 / 12.5 at 400 and 13.6 / 13.3 at
// 640; 64 heads over 32, d_c = 128, 4 sequences 16.8 / 20.5 at 256 and 24.2 / 20.3 at 400.  Over all
// of them a choice costs 0.3% more than the better of the two.
bool mla_window_small_pick(const mla_plan& p, const mla_cache_t& c, int B, MlaWindow win, int kernel) {
  if (!small_shape(p)) return false;
  const mla_config_t& cfg = p.cfg;
  const long long tokens = std::min<long long>(c.T_cap, (long long)win.n_sink + win.window);
  if (tokens > mla::wsmall::kMaxTokens) return false;
  if (kernel == 1) return true;
  const long long ctas = (long long)B * cfg.n_kv_heads;
  const int per_sm = mla::wsmall::layout(cfg).total <= 110 * 1024 ? 2 : 1;
  if (ctas > (long long)per_sm * p.num_sms) return false;
  const int G = cfg.n_heads / cfg.n_kv_heads, units = cfg.d_c / 8;   // (bf16)
  int lanes = 1;
  while (lanes < units && lanes < 32) lanes <<= 1;
  const float us = 6.f + 7e-5f * (G * cfg.head_dim * cfg.d_c) + lanes * (1.6e-3f + 0.5e-3f * G) * tokens;
  return us * (ctas > p.num_sms ? 1.25f : 1.f) <= (kernel == 5 ? 13.f : 20.f);
}

cudaError_t mla_launch_window_small(const mla_plan& p, const mla_cache_t& c, const int32_t* seq_lens, const void* q, int B,
                                    void* out, MlaWindow win, cudaStream_t s) {
  using namespace mla::wsmall;
  const mla_config_t& cfg = p.cfg;
  const Layout L = layout(cfg);
  Args a;
  a.H = cfg.n_heads; a.n_kv = cfg.n_kv_heads; a.d_h = cfg.head_dim; a.r = cfg.r_pairs; a.d_c = cfg.d_c; a.T_cap = c.T_cap;
  a.scale = mla::kLog2e * (cfg.softmax_scale > 0.0f ? cfg.softmax_scale : (float)(1.0 / sqrt((double)cfg.head_dim)));
  a.win = win; a.q = q; a.W_ukF = p.W_ukF; a.W_uv = p.W_uv; a.rope_pair = p.rope_pair; a.theta = p.theta;
  a.seq_lens = seq_lens; a.out = out; a.cache = c; a.err = p.err;
  a.off_uv = L.off_uv; a.off_q = L.off_q; a.off_lat = L.off_lat; a.off_rope = L.off_rope; a.off_p = L.off_p; a.off_part = L.off_part;
  void (*kern)(Args) = nullptr;
  const int G = a.H / a.n_kv;
  if (cfg.dtype == MLA_F32)
    kern = G == 1 ? window_small_kernel<float, 1> : G == 2 ? window_small_kernel<float, 2>
           : G == 3 ? window_small_kernel<float, 3> : window_small_kernel<float, 4>;
  else
    kern = G == 1 ? window_small_kernel<__nv_bfloat16, 1> : G == 2 ? window_small_kernel<__nv_bfloat16, 2>
           : G == 3 ? window_small_kernel<__nv_bfloat16, 3> : window_small_kernel<__nv_bfloat16, 4>;
  cudaError_t e = mla_smem_limit(p, (const void*)kern, L.total);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAttention, false, s);
  if (e == cudaSuccess)
    e = mla_launch_kernel(kern, dim3((unsigned)(B * a.n_kv)), dim3(kThreads), L.total, s, p.opt_pdl, a);
  if (e == cudaSuccess) e = mla_profile_event(p, kProfAttention, true, s);
  return e;
}
