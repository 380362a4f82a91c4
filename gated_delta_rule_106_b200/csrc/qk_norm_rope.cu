// q/k norm + rotary + cache append: per token and head
//   y = x / sqrt(mean(x^2) + eps) * w            (skipped where w is null)
//   pair i of dims [0, R) turns by theta_i = pos_{i mod axes} * inv_freq[i]:
//     (a, b) -> rope_scale * (a cos - b sin, b cos + a sin),
//     (a, b) = dims (i, i + R/2), or (2i, 2i + 1) with `interleaved`
// rounded once: q to q_out, k and (unchanged) v to the token's cache slot.
//
// Angles: the turn theta / 2 pi mod 1 is formed as a 64-bit fixed-point
// product. inv_freq / 2 pi is reduced to its fraction and scaled by 2^64; its
// product with the integer position, modulo 2^64, is the turn's fraction with
// an absolute error below |pos| * 2^-55 turns (the double's own rounding), so
// a position of 10^6 keeps 2^-35 of a turn -- where a 32-bit product
// pos * inv_freq is off by 2^-5 of a radian already. cos and sin then need 32
// bits only.
//
// A CTA takes a few tokens with all their heads, so each (cos, sin) is made
// once for all heads of its token. D / 8 lanes hold a row, 8 elements each.
#include "gdn_common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTok = 4;                 // tokens per CTA

__device__ __forceinline__ float to_f32(const void* w, gdn_dtype t, int i) {
  if (t == GDN_F32) return static_cast<const float*>(w)[i];
  if (t == GDN_F16) return __half2float(static_cast<const __half*>(w)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Round to nearest; finite values past the type's range become its largest,
// NaN stays NaN.
__device__ __forceinline__ float clamp_h(float x) {
  return x != x ? x : fminf(fmaxf(x, -65504.f), 65504.f);
}
__device__ __forceinline__ void put8(__half* p, const float (&f)[8]) {
  uint4 u;
  __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(clamp_h(f[2 * i]), clamp_h(f[2 * i + 1]));
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&f)[8]) { store8(p, f); }

__device__ __forceinline__ float2 turn(double inv_freq, int pos, float scale) {
  double f = inv_freq * 0.15915494309189533577;         // 1 / (2 pi)
  f -= floor(f);
  const uint64_t fixed = __double2ull_rn(f * 18446744073709551616.0);
  const uint64_t a = fixed * (uint64_t)(int64_t)pos;    // mod one turn
  const float half_turns = (float)(int)(a >> 32) * 0x1p-31f;   // in [-1, 1)
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, s * scale);
}

template <class Tx, class To, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs p, int tok) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPW = 32 / LPR;            // rows per warp
  extern __shared__ float2 cs[];           // [tok][R / 2]
  __shared__ float stage[kWarps][256];     // rows being turned
  __shared__ int64_t k_at[kMaxTok], v_at[kMaxTok];
  __shared__ int live_at[kMaxTok];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / LPR, l = lane % LPR;
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  const int half = p.rope_dims >> 1;
  for (int i = tid; i < tok * half; i += kThreads) {
    const int tt = i / half, j = i % half;
    const int64_t t = t0 + tt;
    if (t < p.T)
      cs[i] = turn(p.inv_freq[j], p.positions[(int64_t)(j % p.axes) * p.T + t], p.rope_scale);
  }
  if (tid < tok) {
    const int64_t t = t0 + tid;
    int64_t slot = -1;
    if (t < p.T) slot = p.slot_map ? p.slot_map[t] : t;
    const bool ok = slot >= 0 && slot < (int64_t)p.num_pages * p.page_size;
    // without a cache (queries alone) only the map's sign marks padding
    const bool live = t < p.T && (p.k ? ok : slot >= 0);
    live_at[tid] = live;
    if (live && p.k) {
      const int64_t page = slot / p.page_size, off = slot % p.page_size;
      k_at[tid] = page * p.ks.page + off * p.ks.token;
      v_at[tid] = page * p.vs.page + off * p.vs.token;
    }
  }
  __syncthreads();
  const int Hq = p.q ? p.Hq : 0, Hkv = p.k ? p.Hkv : 0;
  const int H = Hq + 2 * Hkv, rows = tok * H;
  float* row = stage[warp] + sub * D;
  for (int r0 = warp * RPW; r0 < rows; r0 += kWarps * RPW) {
    const int r = r0 + sub;
    const int tt = min(r, rows - 1) / H, hh = min(r, rows - 1) % H;
    const int64_t t = t0 + tt;
    const bool live = r < rows && live_at[tt];
    const int kind = hh < Hq ? 0 : (hh < Hq + Hkv ? 1 : 2);     // q, k, v
    const int h = kind == 0 ? hh : (kind == 1 ? hh - Hq : hh - Hq - Hkv);
    const Tx* src = kind == 0 ? static_cast<const Tx*>(p.q) + t * p.q_row_stride
                  : kind == 1 ? static_cast<const Tx*>(p.k) + t * p.k_row_stride
                              : static_cast<const Tx*>(p.v) + t * p.v_row_stride;
    Raw8<Tx> raw;
    raw.zero();
    if (live) raw.load(src + (int64_t)h * D + l * 8);
    float x[8];
    raw.to_f32(x);
    const void* w = kind == 0 ? p.q_norm_w : p.k_norm_w;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (kind != 2 && w) {
      const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * to_f32(w, p.w_dtype, l * 8 + i);
    }
    if (half) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const int d = l * 8 + i;
          if (kind != 2 && live && d < p.rope_dims) {
            const float2 a = cs[tt * half + (d >> 1)];
            const float u = x[i], v = x[i + 1];
            x[i] = u * a.x - v * a.y;
            x[i + 1] = v * a.x + u * a.y;
          }
        }
      } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) row[l * 8 + i] = x[i];
        __syncwarp();
        if (kind != 2 && live) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = l * 8 + i;
            if (d < half) {
              const float2 a = cs[tt * half + d];
              x[i] = x[i] * a.x - row[d + half] * a.y;
            } else if (d < p.rope_dims) {
              const float2 a = cs[tt * half + d - half];
              x[i] = x[i] * a.x + row[d - half] * a.y;
            }
          }
        }
      }
    }
    if (!live) continue;
    To* dst = kind == 0 ? static_cast<To*>(p.q_out) + (t * p.Hq + h) * D
            : kind == 1 ? static_cast<To*>(p.k_cache) + k_at[tt] + h * p.ks.head
                        : static_cast<To*>(p.v_cache) + v_at[tt] + h * p.vs.head;
    put8(dst + l * 8, x);
  }
}

// Rotary frequencies: f_i = base^(-2i / R). With factor > 1 either all are
// divided by it (context = 0), or each by parts: a pair that makes r_i =
// context * f_i / 2 pi turns over the original context keeps the share
// clamp((r_i - beta_slow) / (beta_fast - beta_slow), 0, 1) of its frequency
// and has the rest divided.
__global__ void rope_inv_freq_kernel(int pairs, double log2_base, double factor, double context,
                                     double beta_fast, double beta_slow, double* out) {
  const int i = threadIdx.x;
  if (i >= pairs) return;
  const double f = exp2(-((double)i / pairs) * log2_base);
  double keep = 0.0;
  if (context > 0.0) {
    const double r = context * f * 0.15915494309189533577;
    keep = fmin(fmax((r - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
  }
  out[i] = f * (keep + (1.0 - keep) / factor);
}

template <class Tx, class To>
cudaError_t launch_typed(const NormRopeArgs& a, unsigned grid, int tok, size_t smem) {
  if (a.D == 256) qk_norm_rope_kernel<Tx, To, 256><<<grid, kThreads, smem, a.stream>>>(a, tok);
  else if (a.D == 128) qk_norm_rope_kernel<Tx, To, 128><<<grid, kThreads, smem, a.stream>>>(a, tok);
  else qk_norm_rope_kernel<Tx, To, 64><<<grid, kThreads, smem, a.stream>>>(a, tok);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a) {
  if (a.T == 0) return cudaSuccess;
  const int tok = a.T > 4 * 148 ? kMaxTok : 1;
  const unsigned grid = (unsigned)((a.T + tok - 1) / tok);
  const size_t smem = (size_t)tok * (a.rope_dims / 2) * sizeof(float2);
  const bool h = a.out_dtype == GDN_F16;
  if (a.x_dtype == GDN_F32)
    return h ? launch_typed<float, __half>(a, grid, tok, smem)
             : launch_typed<float, __nv_bfloat16>(a, grid, tok, smem);
  if (a.x_dtype == GDN_F16)
    return h ? launch_typed<__half, __half>(a, grid, tok, smem)
             : launch_typed<__half, __nv_bfloat16>(a, grid, tok, smem);
  return h ? launch_typed<__nv_bfloat16, __half>(a, grid, tok, smem)
           : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, grid, tok, smem);
}

cudaError_t launch_rope_inv_freq(int rope_dims, double base, double factor, double context,
                                 double beta_fast, double beta_slow, double* out,
                                 cudaStream_t stream) {
  if (rope_dims == 0) return cudaSuccess;
  rope_inv_freq_kernel<<<1, 128, 0, stream>>>(rope_dims / 2, log2(base), factor, context,
                                              beta_fast, beta_slow, out);
  return cudaGetLastError();
}

}  // namespace gdn
