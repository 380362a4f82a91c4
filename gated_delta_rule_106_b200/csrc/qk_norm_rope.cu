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
// pos * inv_freq is off by 2^-5 of a radian already. Its top 32 bits go to fp32, which
// keeps 24 of them: another 2^-26 turns at most (10^-7 of a radian, what cos and sin in
// fp32 are off by anyway, and far below the outputs' 16 bits).
//
// A warp takes a token and a share of its heads (all of them where there are
// tokens enough to fill the chip). D / 8 lanes hold a row, 8 elements each, so a
// lane meets the same dims in every head: it makes its (cos, sin) and loads its
// weights once and keeps them in registers, while several rows are in flight.
// There is no barrier. The share's rows are called into L2 before the angles are
// made.
//
// Bytes bound it at length (32768 tokens of 24 / 4 heads of 256: 186 to 197 us, 5.5 to
// 5.8 TB/s, 83 to 88 % of the copy rate; through shared memory, R = 20, 242 us), issue
// (48 % of the cycles) and the latency of its loads at 8192 (56 us for 41 us of bytes:
// 2.8 waves of warps, 20 per SM at 96 registers); a step of 64 tokens takes 3.9 us. A
// CTA per four tokens with angles and rows in shared memory took 130 us at 8192, one
// kernel for all layouts 63 (see Partner). With 16-bit inputs and D = 256 the kLane
// kernel spills one register.
#include "gdn_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 64;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float to_f32(const void* w, gdn_dtype t, int i) {
  if (t == GDN_F32) return static_cast<const float*>(w)[i];
  if (t == GDN_F16) return __half2float(static_cast<const __half*>(w)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Round to nearest; values past the type's range become its largest, NaN stays
// NaN.
__device__ __forceinline__ void put8(__half* p, const float2 (&f)[4]) {
  uint4 u;
  uint32_t* h = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(f[i].y), "f"(f[i].x));
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float2 (&f)[4]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[i].x, f[i].y);
  *reinterpret_cast<uint4*>(p) = u;
}

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

// How a lane finds the partner of dim d, which decides the registers it needs
// (one kernel for all held 123 and reached 5.2 TB/s at 32768 tokens; 96 without
// the staged exchange and 5.6): adjacent pairs are its own; in the half layout
// the partner is d +- R / 2, the same element of another lane where R / 2 is a
// multiple of 8, else through shared memory.
enum Partner { kOwn, kLane, kStaged };

// What a lane keeps for its token: (cos, sin) of its dims, 8 in the half layout
// (the sine with its side's sign), 4 pairs in the other.
struct Turns { float2 cs[8]; };

// Heads h0 .. h1-1 of one kind (0: q, 1: k, 2: v) of the token by a warp.
template <int KIND, Partner PARTNER, class Tx, class To, int D>
__device__ __forceinline__ void do_heads(const NormRopeArgs& p, const Tx* src, To* dst,
                                         int64_t dst_head, int h0, int h1, const Turns& turns,
                                         float* stage, int lane) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int U = 2;                     // passes in flight
  const int sub = lane / LPR, l = lane % LPR;
  const int half = p.rope_dims >> 1;
  const bool turned = KIND != 2 && l * 8 < p.rope_dims;
  const int from = sub * LPR + (l * 8 < half ? l + half / 8 : l - half / 8);
  const void* weight = KIND == 0 ? p.q_norm_w : p.k_norm_w;
  src += l * 8;
  dst += l * 8;
  Raw8<Tx> raw[U];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u * RPW + sub < h1) raw[u].load_late(src + (int64_t)(h + u * RPW + sub) * D);
      else raw[u].zero();
    }
  };
  load(h0);
  float2 w[4];
  if (KIND != 2 && weight) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = make_float2(to_f32(weight, p.w_dtype, l * 8 + 2 * i),
                         to_f32(weight, p.w_dtype, l * 8 + 2 * i + 1));
  }
  for (int h = h0; h < h1; h += U * RPW) {
    float2 x[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8];
      raw[u].to_f32(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[u][i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
    if (h + U * RPW < h1) load(h + U * RPW);
    if (KIND != 2 && weight) {
      float ss[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 t = __fmul2_rn(x[u][0], x[u][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) t = __ffma2_rn(x[u][i], x[u][i], t);
        ss[u] = t.x + t.y;
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float inv = rsqrtf(ss[u] * (1.0f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[u][i] = __fmul2_rn(__fmul2_rn(x[u][i], make_float2(inv, inv)), w[i]);
      }
    }
    if (KIND != 2 && half) {
      if constexpr (PARTNER == kOwn) {
        if (turned) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // a lane's last pairs may lie behind rope_dims: an infinite value there
              // must not meet the other's sine of 0
              const float2 c = turns.cs[i], v = x[u][i];
              if (l * 4 + i < half)
                x[u][i] = make_float2(v.x * c.x - v.y * c.y, v.y * c.x + v.x * c.y);
            }
        }
      } else {
        float2 other[U][4];
        if constexpr (PARTNER == kLane) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              other[u][i] = make_float2(__shfl_sync(0xffffffffu, x[u][i].x, from & 31),
                                        __shfl_sync(0xffffffffu, x[u][i].y, from & 31));
        } else {
          float* row = stage + sub * D;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float2*>(row + l * 8 + 2 * i) = x[u][i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int d = l * 8 + 2 * i;
              other[u][i].x = d < p.rope_dims ? row[d < half ? d + half : d - half] : 0.f;
              other[u][i].y =
                  d + 1 < p.rope_dims ? row[d + 1 < half ? d + 1 + half : d + 1 - half] : 0.f;
            }
          }
        }
        if (turned) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 a = turns.cs[2 * i], b = turns.cs[2 * i + 1];
              x[u][i] = __ffma2_rn(other[u][i], make_float2(a.y, b.y),
                                   __fmul2_rn(x[u][i], make_float2(a.x, b.x)));
            }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = h + u * RPW + sub;
      if (at < h1) put8(dst + at * dst_head, x[u]);
    }
  }
}

template <Partner PARTNER, class Tx, class To, int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeArgs p, int shares,
                                                                int share_passes) {
  constexpr int LPR = D / 8;               // lanes per row
  constexpr int RPW = 32 / LPR;            // rows per warp and pass
  __shared__ __align__(8) float stage[kWarps][256];     // angles, then rows being turned
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR;
  const int64_t task = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = task / shares;
  let_next_start();
  if (t >= p.T) return;
  const int Hq = p.q ? p.Hq : 0, Hkv = p.k ? p.Hkv : 0;
  // passes of RPW heads: first those of q, then k, then v
  const int pq = (Hq + RPW - 1) / RPW, pkv = (Hkv + RPW - 1) / RPW;
  const int a = (int)(task - t * shares) * share_passes, b = a + share_passes;
  const int q0 = a * RPW, q1 = min(b * RPW, Hq);
  const int k0 = max(a - pq, 0) * RPW, k1 = min((b - pq) * RPW, Hkv);
  const int v0 = max(a - pq - pkv, 0) * RPW, v1 = min((b - pq - pkv) * RPW, Hkv);
  const Tx* q = static_cast<const Tx*>(p.q) + t * p.q_row_stride;
  const Tx* k = static_cast<const Tx*>(p.k) + t * p.k_row_stride;
  const Tx* v = static_cast<const Tx*>(p.v) + t * p.v_row_stride;
  // the whole share is on its way while the angles are made
  auto prefetch = [&](const Tx* x, int h0, int h1) {
    const char* at = reinterpret_cast<const char*>(x + (int64_t)h0 * D);
    const int bytes = (h1 - h0) * D * (int)sizeof(Tx);
    for (int i = lane * 128; i < bytes; i += 32 * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at + i));
  };
  wait_for_previous();
  prefetch(q, q0, q1);
  prefetch(k, k0, k1);
  prefetch(v, v0, v1);

  const int64_t slot = p.slot_map ? p.slot_map[t] : t;
  // without a cache (queries alone) only the map's sign marks padding
  if (slot < 0 || (p.k && slot >= (int64_t)p.num_pages * p.page_size)) return;
  int64_t page = 0, in_page = 0;
  if (p.k) {
    page = (uint32_t)slot / (uint32_t)p.page_size;      // slots are below 2^31
    in_page = slot - page * p.page_size;
  }

  const int half = p.rope_dims >> 1;
  Turns turns;
#pragma unroll
  for (int i = 0; i < 8; ++i) turns.cs[i] = make_float2(1.f, 0.f);
  if (half) {
    // each angle once per warp, a pair per lane and turn
    float2* cs = reinterpret_cast<float2*>(stage[warp]);
    const int pos0 = p.positions[t];
    const int pos1 = p.axes == 3 ? p.positions[p.T + t] : pos0;
    const int pos2 = p.axes == 3 ? p.positions[2 * p.T + t] : pos0;
    for (int j = lane; j < half; j += 32) {
      const int axis = j % 3;
      cs[j] = turn(p.inv_freq[j], axis == 0 ? pos0 : (axis == 1 ? pos1 : pos2), p.rope_scale);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = l * 8 + i;
      if constexpr (PARTNER == kOwn) {
        if (i < 4 && l * 4 + i < half) turns.cs[i] = cs[l * 4 + i];
      } else if (d < p.rope_dims) {
        turns.cs[i] = cs[d < half ? d : d - half];
        if (d < half) turns.cs[i].y = -turns.cs[i].y;
      }
    }
    __syncwarp();
  }

  if (q0 < q1)
    do_heads<0, PARTNER, Tx, To, D>(p, q, static_cast<To*>(p.q_out) + t * p.Hq * D, D, q0, q1, turns,
                           stage[warp], lane);
  if (k0 < k1)
    do_heads<1, PARTNER, Tx, To, D>(p, k,
                           static_cast<To*>(p.k_cache) + page * p.ks.page + in_page * p.ks.token,
                           p.ks.head, k0, k1, turns, stage[warp], lane);
  if (v0 < v1)
    do_heads<2, PARTNER, Tx, To, D>(p, v,
                           static_cast<To*>(p.v_cache) + page * p.vs.page + in_page * p.vs.token,
                           p.vs.head, v0, v1, turns, stage[warp], lane);
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

template <Partner PARTNER, class Tx, class To>
cudaError_t launch_typed(const NormRopeArgs& a) {
  const int rpw = 32 / (a.D / 8);          // rows per warp and pass
  const int passes = ((a.q ? a.Hq : 0) + rpw - 1) / rpw + 2 * (((a.k ? a.Hkv : 0) + rpw - 1) / rpw);
  // shares of a token's heads until there are warps for every SM, a pass at least
  int64_t shares = (148 * 16 + a.T - 1) / a.T;
  if (shares > passes) shares = passes;
  const int share_passes = (int)((passes + shares - 1) / shares);
  shares = (passes + share_passes - 1) / share_passes;
  const unsigned grid = (unsigned)((a.T * shares + kWarps - 1) / kWarps);
  const int s = (int)shares;
  auto kernel = a.D == 256 ? qk_norm_rope_kernel<PARTNER, Tx, To, 256>
              : a.D == 128 ? qk_norm_rope_kernel<PARTNER, Tx, To, 128>
                           : qk_norm_rope_kernel<PARTNER, Tx, To, 64>;
  return launch_early(kernel, dim3(grid), kThreads, 0, a.stream, a, s, share_passes);
}

template <class Tx, class To>
cudaError_t launch_layout(const NormRopeArgs& a) {
  if (a.interleaved || a.rope_dims == 0) return launch_typed<kOwn, Tx, To>(a);
  return a.rope_dims % 16 == 0 ? launch_typed<kLane, Tx, To>(a) : launch_typed<kStaged, Tx, To>(a);
}
template <class Tx>
cudaError_t launch_out(const NormRopeArgs& a) {
  return a.out_dtype == GDN_F16 ? launch_layout<Tx, __half>(a)
                                : launch_layout<Tx, __nv_bfloat16>(a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a) {
  if (a.T == 0) return cudaSuccess;
  if (a.x_dtype == GDN_F32) return launch_out<float>(a);
  return a.x_dtype == GDN_F16 ? launch_out<__half>(a) : launch_out<__nv_bfloat16>(a);
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
