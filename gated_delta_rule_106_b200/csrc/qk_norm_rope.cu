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
// A warp takes a token and a share of its heads (all of them where there are
// tokens enough to fill the chip). D / 8 lanes hold a row, 8 elements each, so a
// lane meets the same dims in every head: it makes its (cos, sin) and loads its
// weights once and keeps them in registers, while several rows are in flight.
// There is no barrier.
#include "gdn_common.cuh"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

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
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs p, int shares,
                                                                int share_rows) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPW = 32 / LPR;            // rows per warp and pass
  constexpr int U = sizeof(Tx) == 4 ? 2 : 4;       // passes in flight
  __shared__ float stage[kWarps][256];     // rows being turned, see below
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, l = lane % LPR;
  const int64_t task = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = task / shares;
  if (t >= p.T) return;
  const int Hq = p.q ? p.Hq : 0, Hkv = p.k ? p.Hkv : 0, H = Hq + 2 * Hkv;
  const int first = (int)(task - t * shares) * share_rows, end = min(first + share_rows, H);

  const int64_t slot = p.slot_map ? p.slot_map[t] : t;
  // without a cache (queries alone) only the map's sign marks padding
  if (slot < 0 || (p.k && slot >= (int64_t)p.num_pages * p.page_size)) return;
  int64_t page = 0, in_page = 0;
  if (p.k) {
    page = (uint32_t)slot / (uint32_t)p.page_size;      // slots are below 2^31
    in_page = slot - page * p.page_size;
  }
  struct Row { int kind, h; };             // 0: q, 1: k, 2: v
  auto row_of = [&](int r) {
    return r < Hq ? Row{0, r} : (r < Hq + Hkv ? Row{1, r - Hq} : Row{2, r - Hq - Hkv});
  };
  auto source = [&](const Row& w) {
    const Tx* src = w.kind == 0 ? static_cast<const Tx*>(p.q) + t * p.q_row_stride
                  : w.kind == 1 ? static_cast<const Tx*>(p.k) + t * p.k_row_stride
                                : static_cast<const Tx*>(p.v) + t * p.v_row_stride;
    return src + (int64_t)w.h * D + l * 8;
  };
  Raw8<Tx> raw[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r < end) raw[u].load(source(row_of(r)));
      else raw[u].zero();
    }
  };
  load(first);

  // (cos, sin) of this lane's dims: 8 in the half layout, 4 pairs in the other
  const int half = p.rope_dims >> 1;
  float2 cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = make_float2(1.f, 0.f);
  if (l * 8 < p.rope_dims) {
    const int pos0 = p.positions[t];
    const int pos1 = p.axes == 3 ? p.positions[p.T + t] : pos0;
    const int pos2 = p.axes == 3 ? p.positions[2 * p.T + t] : pos0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = l * 8 + i;
      if (p.interleaved ? i < 4 && l * 4 + i < half : d < p.rope_dims) {
        const int pair = p.interleaved ? l * 4 + i : (d < half ? d : d - half);
        const int axis = pair % 3;
        cs[i] = turn(p.inv_freq[pair], axis == 0 ? pos0 : (axis == 1 ? pos1 : pos2),
                     p.rope_scale);
        // the half layout adds the partner's sine with the side's sign
        if (!p.interleaved && d < half) cs[i].y = -cs[i].y;
      }
    }
  }

  float w[8];
  int w_kind = -1;
  float* row = stage[warp] + sub * D;
  for (int r0 = first; r0 < end; r0 += U * RPW) {
    Raw8<Tx> now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = raw[u];
    if (r0 + U * RPW < end) load(r0 + U * RPW);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW + sub;
      if (r0 + u * RPW >= end) break;              // the same for the warp
      const bool live = r < end;
      const Row at = row_of(min(r, end - 1));
      float x[8];
      now[u].to_f32(x);
      const void* weight = at.kind == 0 ? p.q_norm_w : p.k_norm_w;
      if (at.kind != w_kind && at.kind != 2) {
        w_kind = at.kind;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight ? to_f32(weight, p.w_dtype, l * 8 + i) : 1.f;
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (at.kind != 2 && weight) {
        const float inv = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
      }
      if (half) {
        if (p.interleaved) {
          if (at.kind != 2 && l * 8 < p.rope_dims) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = a * cs[i].x - b * cs[i].y;
              x[2 * i + 1] = b * cs[i].x + a * cs[i].y;
            }
          }
        } else {
          // the partner of dim d is d + half or d - half: with half a multiple of
          // 8 the same element of another lane, else through shared memory
          float other[8];
          if (half % 8 == 0) {
            const int from = sub * LPR + (l * 8 < half ? l + half / 8 : l - half / 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], from & 31);
          } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) row[l * 8 + i] = x[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int d = l * 8 + i;
              other[i] = d < p.rope_dims ? row[d < half ? d + half : d - half] : 0.f;
            }
          }
          if (at.kind != 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (l * 8 + i < p.rope_dims) x[i] = x[i] * cs[i].x + other[i] * cs[i].y;
          }
        }
      }
      if (!live) continue;
      To* dst = at.kind == 0 ? static_cast<To*>(p.q_out) + (t * p.Hq + at.h) * D
              : at.kind == 1
                  ? static_cast<To*>(p.k_cache) + page * p.ks.page + in_page * p.ks.token +
                        at.h * p.ks.head
                  : static_cast<To*>(p.v_cache) + page * p.vs.page + in_page * p.vs.token +
                        at.h * p.vs.head;
      put8(dst + l * 8, x);
    }
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
cudaError_t launch_typed(const NormRopeArgs& a) {
  const int H = (a.q ? a.Hq : 0) + 2 * (a.k ? a.Hkv : 0);
  const int rpw = 32 / (a.D / 8);          // rows per warp and pass
  const int passes = (H + rpw - 1) / rpw;
  // shares of a token's heads until there are warps for every SM, a pass at least
  int64_t shares = (148 * 16 + a.T - 1) / a.T;
  if (shares > passes) shares = passes;
  const int share_rows = (int)((passes + shares - 1) / shares) * rpw;
  shares = (H + share_rows - 1) / share_rows;
  const unsigned grid = (unsigned)((a.T * shares + kWarps - 1) / kWarps);
  const int s = (int)shares;
  if (a.D == 256)
    qk_norm_rope_kernel<Tx, To, 256><<<grid, kThreads, 0, a.stream>>>(a, s, share_rows);
  else if (a.D == 128)
    qk_norm_rope_kernel<Tx, To, 128><<<grid, kThreads, 0, a.stream>>>(a, s, share_rows);
  else
    qk_norm_rope_kernel<Tx, To, 64><<<grid, kThreads, 0, a.stream>>>(a, s, share_rows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a) {
  if (a.T == 0) return cudaSuccess;
  const bool h = a.out_dtype == GDN_F16;
  if (a.x_dtype == GDN_F32) return h ? launch_typed<float, __half>(a)
                                     : launch_typed<float, __nv_bfloat16>(a);
  if (a.x_dtype == GDN_F16) return h ? launch_typed<__half, __half>(a)
                                     : launch_typed<__half, __nv_bfloat16>(a);
  return h ? launch_typed<__nv_bfloat16, __half>(a)
           : launch_typed<__nv_bfloat16, __nv_bfloat16>(a);
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
