// Attention of one new token per sequence over a paged key-value cache:
//   o_h = sum_j softmax_j(scale * q_h . k_j) v_j,  j < kv_lens[n],
// row j of sequence n at page table[n][j / page_size], offset j % page_size.
//
// The K and V rows cross HBM once, so bytes bound it (2 * G FLOP per cached
// byte for a group of G query heads, a few percent of the tensor rate). The work
// is cut evenly: the units are (sequence, key-value head, block of 64 or 128 tokens) in
// that order, the grid is as many CTAs as fit on the chip at once, and CTA c
// takes units [c U / C, (c + 1) U / C) whatever sequences they belong to. So
// one long sequence spreads over all SMs, and ragged lengths leave none idle;
// the host needs no lengths (every CTA sums kv_lens itself).
//
// In a CTA two warps copy, one the K and one the V rows: they look up each
// row's page and have it copied to shared memory (16-byte cp.async to rows padded
// by 16 bytes, so ldmatrix meets no bank conflict), kStages blocks ahead and
// across sequence ends. Row-sized bulk copies (cp.async.bulk of 2 D bytes) need
// fewer instructions but the lanes of a warp issue them one after the other,
// ~70 cycles each: 2.07 ms against XXX ms for 256 sequences of 4097
// tokens. Four warps compute, 16 tokens of the block each, on mma.sync m16n8k16:
//   S^T = K Q^T   (16 tokens x 8 heads), then
//   O^T += V^T P^T (D x 8 heads), P^T turned in registers by movmatrix.
// Tokens or head dims fill the 16 rows and the group's heads the 8 columns, so
// a group of up to 8 heads wastes no rows. Each warp keeps its own running max
// and sum in fp32 and rescales only when a score passes the max by 8 (2^8).
// P goes in as high and low 16-bit parts: what rounding it once would cost
// (2^-9 relative for bf16) is as much as the output's own rounding, and the
// tensor pipe has room. The warps' pieces of a sequence meet in the block's
// own shared memory at its end. Sequences cut between CTAs leave un-normalised
// pieces (max, sum, O) in the workspace; a second small kernel joins them in
// CTA order.
#include <atomic>

#include "gdn_common.cuh"
#include "launch.h"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kCWarps = 4;                  // computing warps
constexpr int kMaxCtas = 512;
constexpr uint64_t kLimitNs = 2000000000ull;

template <int D, int NT>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;     // 16-token tiles per warp and block
  static constexpr int kTok = 16 * kTiles * kCWarps;  // tokens per block
  static constexpr int kHeads = 8 * NT;               // head columns
  static constexpr int kRow = 2 * D + 16;             // bytes per shared-memory row
  static constexpr int kV = kTok * kRow;              // offsets within a stage
  static constexpr int kQ = 2 * kTok * kRow;
  static constexpr int kStage = kQ + kHeads * kRow;
  static constexpr int kPWarps = 4;                   // copying warps, half for K, half for V
  static constexpr int kThreads = 32 * (kCWarps + kPWarps);
  static constexpr int kCtasPerSm = D == 64 && NT == 1 ? 2 : 1;
  static constexpr int kStages = D == 64 && NT == 2 ? 5 : 3;
  static constexpr int kSmem = kStages * kStage;
  static constexpr int kBatch = D == 256 && NT == 2 ? 2 : 4;   // fragments loaded ahead
  static constexpr int kPad = D + 4;                  // floats per head when pieces meet
  static_assert(kCWarps * kHeads * kPad * 4 <= kQ, "pieces meet in a block's K and V rows");
};

enum : int { kFirst = 1, kLast = 2, kEnd = 4 };

struct BlockDesc { int n, g, ntok, flags, piece, pad[3]; };   // piece: -1 or 0 / 1

struct PagedParams {
  PagedDecodeArgs a;
  int G;
  float sl2;               // scale * log2(e)
  int* status;             // workspace word 0
  int* flag;               // [kMaxCtas] what each CTA met: 0, 1 (a wait ran out), 2 (bad input)
  int4* join;              // [kMaxCtas] {n, g, last CTA, 1} for the sequence piece that starts there
  float* ml;               // [kMaxCtas][2][G][2]
  float* po;               // [kMaxCtas][2][G][D]
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes to shared memory; zeros instead (and no read) with real = false
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real = true) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
// arrives on the barrier once this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <class Th>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two floats as 16-bit high parts, and what they leave as 16-bit low parts
__device__ __forceinline__ void split2(float a, float b, __half, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void split2(float a, float b, __nv_bfloat16, uint32_t& hi,
                                       uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ bool len_ok(const PagedDecodeArgs& a, int len) {
  return len >= 0 && (int64_t)len <= (int64_t)a.max_pages * a.page_size;
}
// blocks of TOK tokens; a length out of range has none
template <int TOK>
__device__ __forceinline__ int blocks_of(const PagedDecodeArgs& a, int len) {
  return len_ok(a, len) ? (int)(((int64_t)len + TOK - 1) / TOK) : 0;
}

// four output values of one (sequence, head): gate and round
__device__ __forceinline__ void put_out(const PagedDecodeArgs& a, int64_t row, int n, int h,
                                        int d, float (&y)[4]) {
  if (a.gate) {
    const uint2 u = *reinterpret_cast<const uint2*>(
        static_cast<const __nv_bfloat16*>(a.gate) + n * a.gate_row_stride + (int64_t)h * a.D + d);
    const float2 g0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 g1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    y[0] /= 1.0f + __expf(-g0.x);
    y[1] /= 1.0f + __expf(-g0.y);
    y[2] /= 1.0f + __expf(-g1.x);
    y[3] /= 1.0f + __expf(-g1.y);
  }
  const int64_t at = row * a.D + d;
  if (a.o_dtype == GDN_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at) =
        make_float4(y[0], y[1], y[2], y[3]);
  } else if (a.o_dtype == GDN_F16) {
    __half2* o = reinterpret_cast<__half2*>(static_cast<__half*>(a.o) + at);
    o[0] = __floats2half2_rn(y[0], y[1]);
    o[1] = __floats2half2_rn(y[2], y[3]);
  } else {
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.o) + at);
    o[0] = __floats2bfloat162_rn(y[0], y[1]);
    o[1] = __floats2bfloat162_rn(y[2], y[3]);
  }
}

template <int B>
__device__ __forceinline__ float total(const float (&s)[B][4], int e) {
  float v = s[0][e];
#pragma unroll
  for (int i = 1; i < B; ++i) v += s[i][e];
  return v;
}

constexpr float kLn2 = 0.69314718055994530942f;

template <int D, int NT, class Th>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtasPerSm)
paged_split_kernel(const __grid_constant__ PagedParams p) {
  using C = Cfg<D, NT>;
  constexpr int kTok = C::kTok;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t full[C::kStages], empty[C::kStages], meet;
  __shared__ BlockDesc desc[C::kStages];
  __shared__ int wrong_page[C::kStages][C::kPWarps];    // met by each copying warp
  __shared__ float2 piece_ml[kCWarps][C::kHeads];
  __shared__ int64_t warp_sum[kCWarps + C::kPWarps];
  __shared__ int start_n, start_len, start_g, start_blk, trouble;
  const PagedDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  // the join may take its place on the chip while this runs
  asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 33 * C::kPWarps);
      mbar_init(&empty[i], kCWarps);
    }
    mbar_init(&meet, 32 * kCWarps);
    fence_mbar_init();
    trouble = start_n = start_len = start_g = start_blk = 0;
  }
  // units before each thread's run of sequences
  const int per = (a.N + C::kThreads - 1) / C::kThreads;
  const int n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  const int len0 = n0 < n1 ? a.kv_lens[n0] : 0;     // kept: usually a thread's only one
  int64_t sum = 0;
  bool odd_len = false;
  for (int n = n0, len = len0; n < n1; ++n) {
    if (n > n0) len = a.kv_lens[n];
    sum += blocks_of<kTok>(a, len);
    odd_len |= !len_ok(a, len);
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (odd_len) atomicMax(&trouble, 2);
  int64_t before = incl - sum, U = 0;
#pragma unroll
  for (int w = 0; w < kCWarps + C::kPWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    U += warp_sum[w];
  }
  before *= a.Hkv;
  U *= a.Hkv;
  const int64_t nc = min((int64_t)gridDim.x, U);    // CTAs that have a unit
  const int64_t r0 = c < nc ? c * U / nc : 0, r1 = c < nc ? (c + 1) * U / nc : 0;
  if (r1 > r0 && before <= r0 && r0 < before + sum * a.Hkv) {
    int64_t rem = r0 - before;
    int len = len0;
    for (int n = n0;;) {
      const int64_t nb = blocks_of<kTok>(a, len);
      if (rem < nb * a.Hkv) {
        start_n = n;
        start_len = len;
        start_g = (int)(rem / nb);
        start_blk = (int)(rem % nb);
        break;
      }
      rem -= nb * a.Hkv;
      if (++n == n1) break;                         // only if lengths change during the call
      len = a.kv_lens[n];
    }
  }
  __syncthreads();

  if (warp >= kCWarps) {
    // ------------------------------------------------------------- copies --
    // Even warps copy K rows, odd ones V rows, each an even share of the block;
    // the first also the queries. A row of D values takes D / 8 lanes.
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    constexpr int kRows = 2 * kTok / C::kPWarps, E = kRows / 32;
    const bool is_v = (warp - kCWarps) & 1, lead = warp == kCWarps;
    const int row0 = (warp - kCWarps) / 2 * kRows;
    const Th* cache = static_cast<const Th*>(is_v ? a.v_cache : a.k_cache);
    const PageStrides cs = is_v ? a.vs : a.ks;
    const uint32_t dst0 = smem_u32(sm) + (is_v ? C::kV : 0) +
                          (row0 + lane / LPR) * C::kRow + (lane % LPR) * 16;
    if (tid == 32 * kCWarps) p.join[c] = make_int4(0, 0, 0, 0);
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    // the unit whose rows are looked up: one ahead of the unit being copied, so
    // that the table's latency passes behind the copies
    int n = start_n, g = start_g, blk = start_blk, len = start_len, nb = 0;
    auto measure = [&] {
      len = (int)min((int64_t)max(len, 0), cap);
      nb = (int)(((int64_t)len + kTok - 1) / kTok);
    };
    int page[E], in_page[E];
    auto lookup = [&] {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t t = (uint32_t)blk * kTok + row0 + lane + 32 * e;
        page[e] = -2;                              // no such row
        if (t < (uint32_t)len) {
          const uint32_t j = t / (uint32_t)a.page_size;
          in_page[e] = (int)(t - j * a.page_size);
          page[e] = a.table[(int64_t)n * a.table_row_stride + j];
          if (page[e] < 0 || page[e] >= a.num_pages) page[e] = -1;
        }
      }
    };
    if (r1 > r0) {
      measure();
      lookup();
    }
    bool first = true, bad = false, begins = blk == 0;
    int it = 0;
    for (int64_t u = r0; u < r1; ++it) {
      const int st = it % C::kStages;
      int64_t off[E];
      bool wrong = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        off[e] = page[e] < 0 ? -1 : page[e] * cs.page + in_page[e] * cs.token + g * cs.head;
        wrong |= page[e] == -1;
      }
      bad |= __any_sync(0xffffffffu, wrong);       // a warp's own rows
      const bool last_blk = blk + 1 == nb, last = last_blk || u + 1 == r1;
      BlockDesc b;
      b.n = n;
      b.g = g;
      b.ntok = min(kTok, len - blk * kTok);
      b.flags = (first ? kFirst : 0) | (last ? kLast : 0);
      // whole in this CTA: straight to the output; the piece that a CTA
      // continues goes to slot 0, the one that it starts to slot 1
      b.piece = begins ? (last_blk ? -1 : 1) : 0;
      const int64_t end = u + (nb - blk);          // unit behind this sequence and head
      // on to the next unit
      ++u;
      ++blk;
      if (last_blk) {
        blk = 0;
        begins = true;
        if (++g == a.Hkv && u < r1) {
          g = 0;
          uint32_t any = 0;
          while (!any && n + 1 < a.N) {            // the next sequence with tokens
            const int m = n + 1 + lane;
            len = m < a.N ? a.kv_lens[m] : 0;
            any = __ballot_sync(0xffffffffu, blocks_of<kTok>(a, len) > 0);
            n += any ? __ffs(any) : 32;
          }
          if (!any) u = r1;                        // only if lengths change during the call
          len = __shfl_sync(0xffffffffu, len, __ffs(any) - 1 & 31);
          measure();
        }
      }
      if (u < r1) lookup();
      if (!mbar_wait_bounded(&empty[st], ((it / C::kStages) & 1) ^ 1, kLimitNs)) break;
      const uint32_t dst = dst0 + st * C::kStage;
      // no branch per row, and the shuffles of eight rows ahead of their copies:
      // a lane's turn at a row then costs its instructions, not their latencies
      constexpr int RB = 8;
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += RB * RPI) {
        int64_t o[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const int r = r0 + i * RPI;
          o[i] = __shfl_sync(0xffffffffu, off[r / 32], r % 32 + lane / LPR);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
          cp_async16(dst + (r0 + i * RPI) * C::kRow,
                     cache + max(o[i], (int64_t)0) + (lane % LPR) * 8, o[i] >= 0);
      }
      if (lead && first) {
        const Th* q = static_cast<const Th*>(a.q) + b.n * a.q_row_stride + (int64_t)b.g * p.G * D;
        for (int i = lane; i < p.G * LPR; i += 32)
          cp_async16(smem_u32(sm) + st * C::kStage + C::kQ + (i / LPR) * C::kRow +
                     (i % LPR) * 16, q + i * 8);
      }
      if (lane == 0) {
        if (lead) {
          desc[st] = b;
          if (last && b.piece == 1)
            p.join[c] = make_int4(b.n, b.g, (int)((end * nc - 1) / U), 1);
        }
        wrong_page[st][warp - kCWarps] = bad;
        if (bad) atomicMax(&trouble, 2);
        mbar_arrive(&full[st]);
      }
      cp_async_arrive(&full[st]);
      first = last;
      if (last) bad = false;
    }
    // end mark, then wait for the copies in flight
    const int st = it % C::kStages;
    const bool fine = mbar_wait_bounded(&empty[st], ((it / C::kStages) & 1) ^ 1, kLimitNs);
    if (fine) {
      if (tid == 32 * kCWarps) desc[st].flags = kEnd;
      if (lane == 0) mbar_arrive(&full[st]);
      mbar_arrive(&full[st]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!fine && lane == 0) atomicMax(&trouble, 3);
  } else {
    // ------------------------------------------------------------ compute --
    const int row = lane >> 2, qd = lane & 3;
    const int mj = lane >> 3, mi = lane & 7;
    // ldmatrix row addresses: matrix mj, row mi
    const int tok0 = warp * 16 * C::kTiles;
    const uint32_t k_off = (uint32_t)((tok0 + (mj & 1) * 8 + mi) * C::kRow + (mj >> 1) * 16);
    const uint32_t v_off = (uint32_t)((tok0 + (mj >> 1) * 8 + mi) * C::kRow + (mj & 1) * 16);
    const uint32_t q_off = (uint32_t)(mi * C::kRow + mj * 16);    // two k-steps per load
    const uint32_t smb = smem_u32(sm);
    uint32_t qf[NT][D / 16][2];
    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
    int meets = 0;
    bool dead = false;
    for (int it = 0; !dead; ++it) {
      const int st = it % C::kStages;
      if (!mbar_wait_bounded(&full[st], (it / C::kStages) & 1, kLimitNs)) { dead = true; break; }
      const BlockDesc b = desc[st];
      if (b.flags & kEnd) break;
      const uint32_t base = smb + st * C::kStage;
      if (b.flags & kFirst) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t r[4];
            ldsm4(base + C::kQ + t * 8 * C::kRow + q_off + kk * 64, r);
            qf[t][2 * kk][0] = r[0];
            qf[t][2 * kk][1] = r[1];
            qf[t][2 * kk + 1][0] = r[2];
            qf[t][2 * kk + 1][1] = r[3];
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
          m[t][0] = m[t][1] = -INFINITY;
          l[t][0] = l[t][1] = 0.f;
        }
      }
      const int nt = b.ntok - tok0;            // this warp's tokens (rows behind them are zeros)
      if (nt > 0) {
        // the fragments of all K tiles, then of all V tiles, in batches: one is
        // loaded ahead of the products that use it
        constexpr int TT = C::kTiles, B = C::kBatch, KB = D / 16 / B, NB = TT * KB;
        uint32_t fr[2][B][4];
        auto load = [&](int i) {                   // batch i of 2 NB
          const int tt = i / KB % TT, kb = i % KB;
          const uint32_t at = base + tt * 16 * C::kRow + kb * B * 32;
#pragma unroll
          for (int e = 0; e < B; ++e) {
            if (i < NB) ldsm4(at + k_off + e * 32, fr[i & 1][e]);
            else ldsm4_t(at + C::kV + v_off + e * 32, fr[i & 1][e]);
          }
        };
        load(0);
        float x[TT][NT][4];                        // tokens row, row + 8; heads 2 qd, 2 qd + 1
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          float s[NT][B][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < B; ++e) s[t][e][0] = s[t][e][1] = s[t][e][2] = s[t][e][3] = 0.f;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            load(tt * KB + kb + 1);                // behind the last K batch: the first of V
#pragma unroll
            for (int e = 0; e < B; ++e)
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma16816<Th>(s[t][e], fr[(tt * KB + kb) & 1][e], qf[t][kb * B + e][0],
                             qf[t][kb * B + e][1]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[tt][t][e] = 16 * tt + row + 8 * (e >> 1) < nt ? total(s[t], e) * p.sl2 : -INFINITY;
        }
        uint32_t hi[TT][NT][2], lo[TT][NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float top[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[e] = fmaxf(x[0][t][e], x[0][t][e + 2]);
#pragma unroll
            for (int tt = 1; tt < TT; ++tt) top[e] = fmaxf(top[e], fmaxf(x[tt][t][e], x[tt][t][e + 2]));
          }
          const int h0 = 8 * t + 2 * qd;
          const bool rise = (h0 < p.G && top[0] > m[t][0] + 8.f) ||
                            (h0 + 1 < p.G && top[1] > m[t][1] + 8.f);
          if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mb = top[e];
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 4));
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
              mb = fmaxf(mb, m[t][e]);
              const float f = mb == -INFINITY ? 1.f : ex2(m[t][e] - mb);
              m[t][e] = mb;
              l[t][e] *= f;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[t][j][e] *= f;
                o[t][j][e + 2] *= f;
              }
            }
          }
          // a max of -inf (no finite score yet) must not meet itself
          const float ma = m[t][0] == -INFINITY ? 0.f : m[t][0];
          const float mb = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) {
            const float p0 = ex2(x[tt][t][0] - ma), p1 = ex2(x[tt][t][1] - mb);
            const float p2 = ex2(x[tt][t][2] - ma), p3 = ex2(x[tt][t][3] - mb);
            l[t][0] += p0 + p2;
            l[t][1] += p1 + p3;
            split2(p0, p1, Th(), hi[tt][t][0], lo[tt][t][0]);
            split2(p2, p3, Th(), hi[tt][t][1], lo[tt][t][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              hi[tt][t][e] = transpose8x8(hi[tt][t][e]);
              lo[tt][t][e] = transpose8x8(lo[tt][t][e]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int tt = i / KB, vb = i % KB;
          if (i + 1 < NB) load(NB + i + 1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < B; ++e)
              mma16816<Th>(o[t][vb * B + e], fr[(NB + i) & 1][e], hi[tt][t][0], hi[tt][t][1]);
#pragma unroll
            for (int e = 0; e < B; ++e)
              mma16816<Th>(o[t][vb * B + e], fr[(NB + i) & 1][e], lo[tt][t][0], lo[tt][t][1]);
          }
        }
      }
      if (b.flags & kLast) {
        // the four warps' pieces meet over this block's K and V rows
        uint8_t* stage = sm + st * C::kStage;
        float* mine = reinterpret_cast<float*>(stage) + warp * C::kHeads * C::kPad;
        mbar_arrive(&meet);
        if (!mbar_wait_bounded(&meet, meets & 1, kLimitNs)) { dead = true; break; }
        ++meets;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = l[t][e];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int h = 8 * t + 2 * qd + e;
            if (row == 0) piece_ml[warp][h] = make_float2(m[t][e], v);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              mine[h * C::kPad + 16 * j + row] = o[t][j][e];
              mine[h * C::kPad + 16 * j + row + 8] = o[t][j][e + 2];
            }
          }
        }
        mbar_arrive(&meet);
        if (!mbar_wait_bounded(&meet, meets & 1, kLimitNs)) { dead = true; break; }
        ++meets;
        const float* all = reinterpret_cast<const float*>(stage);
        int bad = 0;
#pragma unroll
        for (int w = 0; w < C::kPWarps; ++w) bad |= wrong_page[st][w];
        for (int i = tid; i < p.G * (D / 4); i += 32 * kCWarps) {
          const int h = i / (D / 4), d = 4 * (i % (D / 4));
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kCWarps; ++w) M = fmaxf(M, piece_ml[w][h].x);
          float L = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < kCWarps; ++w) {
            const float2 ml = piece_ml[w][h];
            const float f = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
            const float4 v = *reinterpret_cast<const float4*>(
                all + (w * C::kHeads + h) * C::kPad + d);
            L += f * ml.y;
            y[0] += f * v.x;
            y[1] += f * v.y;
            y[2] += f * v.z;
            y[3] += f * v.w;
          }
          if (bad) L = __int_as_float(0x7fc00000);
          const int hq = b.g * p.G + h;
          if (b.piece < 0) {
            const float inv = 1.f / L;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= inv;
            put_out(a, (int64_t)b.n * a.Hq + hq, b.n, hq, d, y);
            if (a.lse && d == 0) a.lse[(int64_t)b.n * a.Hq + hq] = (M + log2f(L)) * kLn2;
          } else {
            const int64_t at = ((int64_t)c * 2 + b.piece) * p.G + h;
            *reinterpret_cast<float4*>(p.po + at * D + d) = make_float4(y[0], y[1], y[2], y[3]);
            if (d == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(M, L);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (dead) atomicMax(&trouble, 3);           // a wait ran out: more than bad input
  }
  __syncthreads();
  if (tid == 0) p.flag[c] = trouble == 3 ? 1 : trouble;
}

// Joins the pieces of the sequence (and key-value head) that CTA c of the split
// kernel started and did not end; also sums up what the CTAs met.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p) {
  constexpr int kLanes = D / 4, kParts = kJoinThreads / kLanes;
  __shared__ float weight[kMaxCtas];
  __shared__ float4 acc[kParts][kLanes];
  __shared__ float red[kJoinThreads / 32];
  const PagedDecodeArgs& a = p.a;
  const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // sequences without a token, or with a length out of range: nothing of the
  // split kernel's is needed for them
  for (int n = c; n < a.N; n += gridDim.x) {
    const int len = a.kv_lens[n];
    const bool ok = len_ok(a, len);
    if (ok && len > 0) continue;
    const float v = ok ? 0.f : __int_as_float(0x7fc00000);
    for (int i = tid; i < a.Hkv * (D / 4); i += kJoinThreads) {
      const int hq = i / (D / 4) * p.G + h, d = 4 * (i % (D / 4));
      float y[4] = {v, v, v, v};
      put_out(a, (int64_t)n * a.Hq + hq, n, hq, d, y);
      if (a.lse && d == 0) a.lse[(int64_t)n * a.Hq + hq] = ok ? -INFINITY : v;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c == 0 && h == 0) {
    int f = 0;
    for (int i = tid; i < (int)gridDim.x; i += kJoinThreads) f |= p.flag[i];
    const int timeout = __syncthreads_or(f & 1), wrong = __syncthreads_or(f & 2);
    if (tid == 0) *p.status = timeout ? 1 : (wrong ? 2 : 0);
  }
  const int4 j = p.join[c];
  if (!j.w) return;
  const int pieces = j.z - c + 1;             // at most the grid's CTAs
  auto at = [&](int i) { return ((int64_t)(c + i) * 2 + (i == 0)) * p.G + h; };
  // weights of the pieces: all loads at once, then sums in a fixed order
  float2 ml[kMaxCtas / kJoinThreads];
  float M = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMaxCtas / kJoinThreads; ++k) {
    const int i = tid + k * kJoinThreads;
    ml[k] = i < pieces ? *reinterpret_cast<const float2*>(p.ml + at(i) * 2)
                       : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, ml[k].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[w]);
  float L = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxCtas / kJoinThreads; ++k) {
    const float f = ml[k].x == -INFINITY ? (ml[k].y == 0.f ? 0.f : 1.f) : ex2(ml[k].x - M);
    weight[tid + k * kJoinThreads] = f;
    L += f * ml[k].y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  __syncthreads();
  if (lane == 0) red[warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) L += red[w];
  const int part = tid / kLanes, d = 4 * (tid % kLanes);
  float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = part; i < pieces; i += kParts) {
    const float4 v = *reinterpret_cast<const float4*>(p.po + at(i) * D + d);
    const float f = weight[i];
    y[0] += f * v.x;
    y[1] += f * v.y;
    y[2] += f * v.z;
    y[3] += f * v.w;
  }
  acc[part][tid % kLanes] = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (part) return;
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    const float4 v = acc[i][tid % kLanes];
    y[0] += v.x;
    y[1] += v.y;
    y[2] += v.z;
    y[3] += v.w;
  }
  const float inv = 1.f / L;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] *= inv;
  const int hq = j.y * p.G + h;
  put_out(a, (int64_t)j.x * a.Hq + hq, j.x, hq, d, y);
  if (a.lse && d == 0) a.lse[(int64_t)j.x * a.Hq + hq] = (M + log2f(L)) * kLn2;
}

constexpr size_t kHeadBytes = 256 + kMaxCtas * 4 + kMaxCtas * 16;

template <int D, int NT, class Th>
cudaError_t launch_split(const PagedParams& p, int sms) {
  using C = Cfg<D, NT>;
  static std::atomic<uint64_t> ready{0};      // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(paged_split_kernel<D, NT, Th>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const int grid = min(sms * C::kCtasPerSm, kMaxCtas);
  paged_split_kernel<D, NT, Th><<<grid, C::kThreads, C::kSmem, p.a.stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join starts while the split's last CTAs end, and waits for them
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, (unsigned)p.G);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = p.a.stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, p);
}

template <int D, class Th>
cudaError_t launch_heads(const PagedParams& p, int sms) {
  return p.G <= 8 ? launch_split<D, 1, Th>(p, sms) : launch_split<D, 2, Th>(p, sms);
}
template <class Th>
cudaError_t launch_dim(const PagedParams& p, int sms) {
  if (p.a.D == 256) return launch_heads<256, Th>(p, sms);
  if (p.a.D == 128) return launch_heads<128, Th>(p, sms);
  return launch_heads<64, Th>(p, sms);
}

}  // namespace

size_t paged_decode_workspace(int group, int D) {
  return kHeadBytes + (size_t)kMaxCtas * 2 * group * (D + 2) * 4;
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a) {
  if (a.N == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PagedParams p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.status = reinterpret_cast<int*>(ws);
  p.flag = reinterpret_cast<int*>(ws + 256);
  p.join = reinterpret_cast<int4*>(ws + 256 + kMaxCtas * 4);
  p.po = reinterpret_cast<float*>(ws + kHeadBytes);
  p.ml = p.po + (size_t)kMaxCtas * 2 * p.G * a.D;
  return a.kv_dtype == GDN_F16 ? launch_dim<__half>(p, sms) : launch_dim<__nv_bfloat16>(p, sms);
}

}  // namespace gdn
