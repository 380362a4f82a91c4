// Attention of one new token per sequence over a paged key-value cache:
//   o_h = sum_j softmax_j(scale * q_h . k_j) v_j,  j < kv_lens[n],
// row j of sequence n at page table[n][j / page_size], offset j % page_size.
//
// The K and V rows cross HBM once, so bytes bound it (2 * G FLOP per cached
// byte for a group of G query heads, a few percent of the tensor rate): 256
// sequences of 4097 tokens (24 / 4 heads, D = 256, 4.3 GB) take 665 to 685 us, 6.4
// TB/s, call after call on most B200s, where the power cap holds the clocks at 1.6 GHz,
// and 625 to 630 us, 6.9 TB/s, on one that kept them and elsewhere for the first 50 ms
// after a pause; one sequence of 131071 tokens 88 us, 6.1 TB/s.
//
// The work is cut evenly: the units are (sequence, key-value head, block of 64 or
// 128 tokens) in that order, and CTAs take ranges of units whatever sequences
// they belong to (see Ranges). So one long sequence spreads over all SMs, ragged
// lengths leave none idle, and the host needs no lengths: every CTA sums kv_lens
// itself. The cuts depend on the lengths and the chip alone, never on which CTA
// comes first, so equal calls give equal bits.
//
// In a CTA copying warps fill a ring of three blocks in shared memory, ahead of the
// computing warps and across sequence ends. They look each page up and copy its
// rows by TMA, boxes of rows x 64 dims with the 128-byte swizzle (ldmatrix then
// meets no bank conflict); where pages have no factor of 8 rows, by 16-byte
// cp.async to the same places. What was measured on the way (256 x 4097 tokens):
// row-sized cp.async.bulk 2.07 ms (a warp's lanes issue them one after the other,
// ~70 cycles each), cp.async by two warps 0.80, by four 0.64 (0.80 under the power
// cap: the copies' instructions cost energy), TMA 0.63 (0.67).
//
// Four warps compute, 16-token tiles, on mma.sync m16n8k16 (the legacy warp MMA: a
// tcgen05 tile of 128 rows would be mostly empty, and the tensor pipe is busy in 15 % of
// the cycles at D = 256, 24 / 4 heads):
//   S^T = K Q^T   (16 tokens x 8 heads), then
//   O^T += V^T P^T (D x 8 heads), P^T turned in registers by movmatrix.
// Tokens or head dims fill the 16 rows and the group's heads the 8 columns, so
// a group of up to 8 heads wastes no rows. Each warp keeps its own reference (near
// the running max) and sum in fp32 and rescales rarely (kTop below).
// P goes in as high and low 16-bit parts: what rounding it once would cost
// (2^-9 relative for bf16) is as much as the output's own rounding, and the
// tensor pipe has room. For fp32 outputs bf16 takes a third part
// (1.3e-6 of the output without it, 1e-7 with it). The warps' pieces of a sequence
// meet in the block's own shared memory at its end. Sequences cut between ranges
// leave un-normalised pieces (max, sum, O) in the workspace; a second small kernel
// joins them in order (3 to 4 us).
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "gdn_common.cuh"
#include "launch.h"
#include "pdl.cuh"
#include "sm100.cuh"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kCWarps = 4;                  // computing warps
constexpr int kPhases = 3;                  // see Ranges
constexpr int kMaxBase = 2 * 160;           // CTAs at once
constexpr int kMaxRanges = kPhases * kMaxBase;
constexpr int kAhead = 8;                   // blocks that table entries are called in ahead
// Weights are 2^(score - m) with m 11 below the highest score when it was set, and m
// moves when a score passes it by 15: weights reach 2^15, and fp16's smallest steps
// (2^-24) are 2^-35 of the largest. A long context whose sum is one key's and the
// rest's of 10^5 keys with weights of 2^-20 each needs that.
constexpr float kLift = 11.f, kTop = 15.f;
// Waits of warps for one another have the caller's bound (gdn_set_wait_limit_ns); at
// the end of a CTA that gave up, each stage that may still be written to is waited for
// this long. A copy lands in microseconds; the time passes in full where another warp
// never came to the stage.
constexpr uint64_t kDrainNs = 50000000ull;
constexpr uint64_t kSuspendNs = 1000000ull;

template <int D, int NT>
struct Cfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;     // 16-token tiles per warp and block
  static constexpr int kTok = 16 * kTiles * kCWarps;  // tokens per block
  static constexpr int kHeads = 8 * NT;               // head columns
  // A stage holds the K, then the V rows of a block, each as D / 64 column chunks
  // [kTok rows][128 bytes] whose 16-byte units are permuted within a row as TMA's
  // 128-byte swizzle does: unit j of row r is at j ^ (r % 8).
  static constexpr int kChunk = kTok * 128;
  static constexpr int kV = kTok * 2 * D;
  static constexpr int kStage = 2 * kV;
  static constexpr int kQRow = 2 * D + 16;            // queries behind the stages, padded rows
  static constexpr int kQStage = kHeads * kQRow;
  // copying warps, half for K, half for V: at D = 128 a row is half a warp's copy
  // and its lookup counts more
  static constexpr int kPWarps = D == 128 && NT == 1 ? 8 : 4;
  static constexpr int kThreads = 32 * (kCWarps + kPWarps);
  static constexpr int kRuns = D == 64 ? 64 : 256;      // runs of sequences that are summed
  static constexpr int kCtasPerSm = D == 64 && NT == 1 ? 2 : 1;
  static constexpr int kStages = D == 64 && NT == 2 ? 5 : 3;
  static constexpr int kSmem = 1024 + kStages * (kStage + kQStage);   // 1024 to align
  static constexpr int kBatch = D == 256 && NT == 2 ? 2 : 4;   // fragments loaded ahead
  // floats per head when pieces meet (padded against bank conflicts where there is room)
  static constexpr int kPad = D == 256 && NT == 2 ? D : D + 4;
  // two CTAs per SM: 228 KB with 1 KB of the system's and ~1.5 KB of barriers and sums each
  static_assert(kCtasPerSm == 1 || kSmem + 2560 <= 114 * 1024, "two CTAs fit");
  static_assert(kCWarps * kHeads * kPad * 4 <= kStage, "pieces meet in a block's K and V rows");
};

enum : int { kFirst = 1, kLast = 2, kEnd = 4 };

struct BlockDesc { int n, g, ntok, flags, piece, range, pad[2]; };   // piece: -1 or 0 / 1

// How the U units are cut into ranges, in order: `base` (the CTAs that run at
// once) equal ranges that hold 34 of 40 parts of the work, then base ranges with
// 4 and base with 2 parts, which go to whoever is done: SMs differ by 10 % in the
// bandwidth they get. Below 64 units per CTA the extra pieces cost more than that
// (1 x 131071 tokens, 55 units: 102 us against 94), and there is one phase.
constexpr int kStealUnits = 64;
struct Ranges {
  int64_t U, q;               // U = q * 40 base + r
  int base, phases, r;
  __device__ Ranges(int64_t units, int ctas, bool steal) : U(units), base(ctas), phases(1) {
    if (steal && units >= kStealUnits * (int64_t)ctas) phases = 3;
    else base = max((int)min((int64_t)ctas, units), 1);
    if (units <= INT32_MAX) {
      q = (uint32_t)units / (uint32_t)(40 * base);
    } else {
      q = units / (40 * base);
    }
    r = (int)(units - q * (40 * base));
  }
  // parts of 40 behind phase ph
  __device__ int rest(int ph) const { return ph == 0 ? 40 : (ph >= phases ? 0 : 10 - 4 * ph); }
  // first unit of range v, U * part / (40 base) (U behind the last range)
  __device__ int64_t start(int v) const {
    if (v >= phases * base) return U;
    const int ph = v < base ? 0 : (v < 2 * base ? 1 : 2), i = v - ph * base;
    const int part = (40 - rest(ph)) * base + (rest(ph) - rest(ph + 1)) * i;
    return q * part + (uint32_t)(r * part) / (uint32_t)(40 * base);   // r, part < 40 * 320
  }
  // the range of unit x: the last v with start(v) <= x
  __device__ int of(int64_t x) const {
    const int64_t most = ((x + 1) * 40 * base - 1) / U;
    int ph = 0;
    while (ph + 1 < phases && (int64_t)(40 - rest(ph + 1)) * base <= most) ++ph;
    const int64_t i = (most - (int64_t)(40 - rest(ph)) * base) / (rest(ph) - rest(ph + 1));
    return ph * base + (int)min(i, (int64_t)base - 1);
  }
};

struct PagedParams {
  PagedDecodeArgs a;
  int G;
  float sl2;               // scale * log2(e)
  int* status;             // workspace word 0
  int box;                 // rows per TMA copy, or 0: rows are copied by cp.async
  int copy_warps;          // copying warps at work
  bool k_token_first, v_token_first;    // the order of the maps' middle dimensions
  int base;                // CTAs that run at once; more in the grid are taken over
  uint64_t limit_ns;       // bound of a wait
  bool poll;               // a bound below kSuspendNs
  int* flag;               // [grid] what each CTA met: 0, 1 (a wait ran out), 2 (bad input)
  int4* join;              // [grid] {n, g, last range, 1} for the piece that starts in a range
  float* ml;               // [grid][2][G][2]
  float* po;               // [grid][2][G][D]
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes to shared memory under an L2 policy; zeros instead (and no read)
// with real = false
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real,
                                           uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(real ? 16 : 0), "l"(policy)
               : "memory");
}
// Box at column x, (y, z) = (head, token) or (token, head) and page of a cache.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                        int page, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(page),
      "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// Waits for at most p.limit_ns. A try_wait may suspend its warp for longer than a read of
// global memory takes (a suspend-time operand did not change that): short bounds are
// polled for.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, const PagedParams& p) {
  auto look = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (look()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (p.poll ? look() : mbar_try_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > p.limit_ns) return false;
  }
}
// The same answer in all lanes, so that a warp leaves its loop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const PagedParams& p) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, p));
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// arrives on the barrier once this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Asks the hardware for a CTA of this grid that has not started; the answer
// (16 bytes) lands on `bar`.
__device__ __forceinline__ void ask_cta(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(smem_u32(answer)), "r"(smem_u32(bar))
      : "memory");
}
// The CTA that the answer gives us, or -1: none is left.
__device__ __forceinline__ int given_cta(const uint4* answer) {
  int id;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(id)
      : "r"(smem_u32(answer))
      : "memory");
  return id;
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
// two floats rounded to 16 bits; a and b keep what that leaves
__device__ __forceinline__ uint32_t take2(float& a, float& b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  a -= f.x;
  b -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t take2(float& a, float& b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  a -= f.x;
  b -= f.y;
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ bool len_ok(const PagedDecodeArgs& a, int len) {
  return len >= 0 && (int64_t)len <= (int64_t)a.max_pages * a.page_size;
}
// blocks of TOK tokens; a length out of range has none
template <int TOK>
__device__ __forceinline__ int blocks_of(const PagedDecodeArgs& a, int len) {
  return len_ok(a, len) ? (int)(((int64_t)len + TOK - 1) / TOK) : 0;
}

// The gate of V = 2 or 4 values of one (sequence, head).
template <int V> struct Gate { __nv_bfloat162 v[V / 2]; };
template <int V>
__device__ __forceinline__ Gate<V> load_gate(const PagedDecodeArgs& a, int n, int h, int d) {
  Gate<V> g;
  if (a.gate) {
    const __nv_bfloat162* src = reinterpret_cast<const __nv_bfloat162*>(
        static_cast<const __nv_bfloat16*>(a.gate) + n * a.gate_row_stride + (int64_t)h * a.D + d);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) g.v[i] = __ldcg(src + i);   // read once, see the join
  }
  return g;
}
// V output values of one (sequence, head) row: gate and round
template <int V>
__device__ __forceinline__ void put_out(const PagedDecodeArgs& a, int64_t row, int d,
                                        const Gate<V>& gate, float (&y)[V]) {
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = __bfloat1622float2(gate.v[i]);
      y[2 * i] = __fdividef(y[2 * i], 1.0f + __expf(-v.x));        // within 2 ulp
      y[2 * i + 1] = __fdividef(y[2 * i + 1], 1.0f + __expf(-v.y));
    }
  }
  const int64_t at = row * a.D + d;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if (a.o_dtype == GDN_F32)
      *reinterpret_cast<float2*>(static_cast<float*>(a.o) + at + i) = make_float2(y[i], y[i + 1]);
    else if (a.o_dtype == GDN_F16)
      *reinterpret_cast<__half2*>(static_cast<__half*>(a.o) + at + i) =
          __floats2half2_rn(y[i], y[i + 1]);
    else
      *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.o) + at + i) =
          __floats2bfloat162_rn(y[i], y[i + 1]);
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
paged_split_kernel(const __grid_constant__ PagedParams p,
                   const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D, NT>;
  constexpr int kTok = C::kTok;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], meet;
  __shared__ BlockDesc desc[C::kStages];
  __shared__ int wrong_page[C::kStages][C::kPWarps];    // met by each copying warp
  __shared__ float2 piece_ml[kCWarps][C::kHeads];
  __shared__ int64_t warp_sum[kCWarps + C::kPWarps];
  __shared__ int64_t run_before[C::kRuns];         // units before each run of sequences
  __shared__ int run_len[C::kRuns];                // length of the run's first sequence
  __shared__ __align__(16) uint4 answer;
  __shared__ uint64_t asked_full, asked_free;
  __shared__ int trouble;
  const PagedDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int copied = 0;                                  // blocks whose copies this warp began

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      // the leading lanes of the copying warps, and each lane's own copies (TMA:
      // the queries' alone, by the first warp)
      mbar_init(&full[i], p.copy_warps + 32 * (p.box ? 1 : C::kPWarps));
      mbar_init(&empty[i], kCWarps);
    }
    mbar_init(&meet, 32 * kCWarps);
    mbar_init(&asked_full, 1);
    mbar_init(&asked_free, p.copy_warps);
    fence_mbar_init();
    trouble = 0;
  }
  if (tid < C::kStages * C::kPWarps) (&wrong_page[0][0])[tid] = 0;
  wait_for_previous();
  const int per = (a.N + C::kRuns - 1) / C::kRuns;  // a run per thread, the first kRuns threads
  const int n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
  const int len0 = n0 < n1 ? a.kv_lens[n0] : 0;
  if (tid < C::kRuns) run_len[tid] = len0;
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
  if (tid < C::kRuns) run_before[tid] = before * a.Hkv;
  U *= a.Hkv;
  const Ranges ranges(U, p.base, (int)gridDim.x > p.base);
  __syncthreads();

  if (warp >= kCWarps) {
    // ------------------------------------------------------------- copies --
    // Even warps copy K rows, odd ones V rows, the first also the queries. With TMA
    // a lane takes a box of rows of one page, and as many warps work as the boxes
    // need (lanes issue one after the other). Else each has an even share of the
    // block's rows, and a row of D values takes D / 8 lanes.
    const bool tma = p.box != 0;
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    constexpr int kRows = 2 * kTok / C::kPWarps, E = kRows / 32;
    const bool is_v = (warp - kCWarps) & 1, lead = warp == kCWarps;
    const int row0 = (warp - kCWarps) / 2 * kRows;
    const Th* cache = static_cast<const Th*>(is_v ? a.v_cache : a.k_cache);
    const PageStrides cs = is_v ? a.vs : a.ks;
    const uint32_t side = smem_u32(sm) + (is_v ? C::kV : 0);
    const uint32_t dst0 = side + (row0 + lane / LPR) * 128 + (lane % LPR) / 8 * C::kChunk +
                          (((lane % 8) ^ (lane / LPR)) << 4);
    const CUtensorMap* map = is_v ? &v_map : &k_map;
    const bool token_first = is_v ? p.v_token_first : p.k_token_first;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    // cached rows are read once: they leave L2 before the table, queries and gates
    uint64_t once;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    // the unit whose rows are looked up, one ahead of the unit being copied, so
    // that the table's latency passes behind the copies: range, units to its end,
    // sequence, key-value head, block; the sequence's length and blocks
    const bool idle = warp - kCWarps >= p.copy_warps;
    const int box_row = ((warp - kCWarps) / 2 + lane * (p.copy_warps / 2)) * p.box;
    int range = blockIdx.x, n = 0, g = 0, blk = 0, len = 0, nb = 0;
    int64_t u = 0, r1 = 0;
    bool first = true, begins = true, bad = false;
    bool steal = (int)gridDim.x > p.base, asked = false, late = false;
    bool answer_due = false;                            // lane 0 of the lead: one is on its way
    int answers = 0;
    auto measure = [&] {
      len = (int)min((int64_t)max(len, 0), cap);
      nb = (int)(((int64_t)len + kTok - 1) / kTok);
    };
    int page[E] = {}, in_page[E];                       // in_page < 0: no such row
    // With the rows of three blocks per SM in flight a read from HBM takes ~5 us;
    // what is needed later is called into L2 before: table entries some blocks
    // ahead, and the gates when their sequence starts.
    auto lookup = [&] {
      if (lead && lane < 2) {
        const int64_t j = ((int64_t)blk + kAhead + 4 * lane) * kTok / a.page_size;
        if (j < a.max_pages) prefetch_l2(a.table + (int64_t)n * a.table_row_stride + j);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t row = tma ? box_row : row0 + lane + 32 * e;
        const uint32_t t = (uint32_t)blk * kTok + row;
        in_page[e] = -1;
        if (t < (uint32_t)len && (!tma || (e == 0 && row < (uint32_t)kTok))) {
          const uint32_t j = t / (uint32_t)a.page_size;
          in_page[e] = (int)(t - j * a.page_size);
          page[e] = a.table[(int64_t)n * a.table_row_stride + j];   // looked at a unit later
        }
      }
    };
    // go to the first unit of `range`
    auto enter = [&] {
      u = ranges.start(range);
      r1 = ranges.start(range + 1);
      if (lead && lane == 0) {
        p.join[range] = make_int4(0, 0, 0, 0);
        if (range != (int)blockIdx.x) p.flag[range] = 0;   // that CTA never starts
      }
      if (u >= r1) return;
      // the last run of sequences that starts at or before u ...
      int at = 0;
#pragma unroll
      for (int k = 0; k < C::kRuns / 32; ++k) at += run_before[lane * (C::kRuns / 32) + k] <= u;
      at = __reduce_add_sync(0xffffffffu, at) - 1;
      // ... and the sequence in it
      int64_t rem = u - run_before[at];
      n = at * per;
      if (per == 1) {
        len = run_len[at];
      } else {
        for (;; n += 32) {
          const int m = n + lane;
          len = m < a.N && m < (at + 1) * per ? a.kv_lens[m] : 0;
          const int64_t units = (int64_t)blocks_of<kTok>(a, len) * a.Hkv;
          int64_t upto = units;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
          }
          const uint32_t past = __ballot_sync(0xffffffffu, upto > rem);
          if (past || n + 32 >= (at + 1) * per) {  // without a hit: lengths change during the call
            const int src = past ? __ffs(past) - 1 : 0;
            rem -= __shfl_sync(0xffffffffu, upto - units, src);
            len = __shfl_sync(0xffffffffu, len, src);
            n = min(n + src, a.N - 1);
            break;
          }
          rem -= __shfl_sync(0xffffffffu, upto, 31);
        }
      }
      measure();
      if (nb == 0) { u = r1; return; }             // lengths change during the call
      if (rem <= INT32_MAX) {
        g = (int)((uint32_t)rem / (uint32_t)nb);
        blk = (int)rem - g * nb;
      } else {
        g = (int)(rem / nb);
        blk = (int)(rem % nb);
      }
      g = min(g, a.Hkv - 1);
      begins = blk == 0;
      first = true;
    };
    auto ask = [&] {
      if (lead && lane == 0) {
        if (answers > 0 && !wait_bounded(&asked_free, (answers - 1) & 1, p)) {
          late = true;
        } else {
          ask_cta(&answer, &asked_full);
          answer_due = true;
        }
      }
      asked = true;
    };
    // when a range is done, take over CTAs that have not started until one has units
    auto refill = [&] {
      while (u >= r1 && steal) {
        if (!asked) ask();
        if (!warp_wait(&asked_full, answers & 1, p)) { late = true; break; }
        range = given_cta(&answer);
        asked = answer_due = false;
        ++answers;
        fence_proxy_async_smem();                  // read here before the next answer lands
        __syncwarp();
        if (lane == 0) mbar_arrive(&asked_free);
        if (range < 0) steal = false;
        else enter();
      }
    };
    if (!idle) {
      enter();
      refill();
      if (u < r1) lookup();
    }
    int it = 0;
    for (; u < r1; ++it) {
      const int st = it % C::kStages;
      int64_t off[E];
      bool wrong = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = in_page[e] >= 0, ok = in && page[e] >= 0 && page[e] < a.num_pages;
        off[e] = ok ? page[e] * cs.page + in_page[e] * cs.token + g * cs.head : -1;
        wrong |= in && !ok;
      }
      bad |= __any_sync(0xffffffffu, wrong);       // a warp's own rows
      const int page_now = page[0], token_now = in_page[0];
      const bool box_now = off[0] >= 0;
      const bool bad_now = bad, first_now = first;
      const bool last_blk = blk + 1 == nb, last = last_blk || u + 1 == r1;
      BlockDesc b;
      b.n = n;
      b.g = g;
      b.ntok = min(kTok, len - blk * kTok);
      b.flags = (first ? kFirst : 0) | (last ? kLast : 0);
      // whole in this range: straight to the output; the piece that a range
      // continues goes to slot 0, the one that it starts to slot 1
      b.piece = begins ? (last_blk ? -1 : 1) : 0;
      b.range = range;
      const int64_t end = u + (nb - blk);          // unit behind this sequence and head
      // on to the next unit; a range's successor is asked for shortly before its end
      ++u;
      ++blk;
      first = last;
      if (last) bad = false;
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
          len = __shfl_sync(0xffffffffu, len, (__ffs(any) - 1) & 31);
          measure();
        }
      }
      if (steal && !asked && r1 - u <= 3) ask();
      refill();
      if (u < r1) lookup();
      if (!warp_wait(&empty[st], ((it / C::kStages) & 1) ^ 1, p)) {
        late = true;
        break;
      }
      if (!tma) {
        // no branch per row, and the shuffles of eight rows ahead of their copies:
        // a lane's turn at a row then costs its instructions, not their latencies
        const uint32_t dst = dst0 + st * C::kStage;
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
            cp_async16((dst ^ (((i * RPI) & 7) << 4)) + (r0 + i * RPI) * 128,
                       cache + max(o[i], (int64_t)0) + (lane % LPR) * 8, o[i] >= 0, once);
        }
      }
      if (lead && first_now) {
        const Th* q = static_cast<const Th*>(a.q) + b.n * a.q_row_stride + (int64_t)b.g * p.G * D;
        for (int i = lane; i < p.G * LPR; i += 32)
          cp_async16(smem_u32(sm) + C::kStages * C::kStage + st * C::kQStage +
                     (i / LPR) * C::kQRow + (i % LPR) * 16, q + i * 8);
        if (a.gate) {
          const char* g = reinterpret_cast<const char*>(
              static_cast<const __nv_bfloat16*>(a.gate) + b.n * a.gate_row_stride +
              (int64_t)b.g * p.G * D);
          for (int i = lane * 128; i < p.G * D * 2; i += 32 * 128) prefetch_l2(g + i);
        }
      }
      if (lane == 0) {
        if (lead) {
          desc[st] = b;
          if (last && b.piece == 1)
            p.join[b.range] = make_int4(b.n, b.g, ranges.of(end - 1), 1);
        }
        wrong_page[st][warp - kCWarps] = bad_now;
        if (bad_now) atomicMax(&trouble, 2);
        if (!tma) mbar_arrive(&full[st]);
      }
      if (!tma || lead) cp_async_arrive(&full[st]);
      if (tma) {
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box_now));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * p.box * 2 * D);
        __syncwarp();
        if (box_now) {
          const uint32_t dst = side + st * C::kStage + box_row * 128;
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_box(dst + x * C::kChunk, map, x * 64, token_first ? token_now : b.g,
                    token_first ? b.g : token_now, page_now, &full[st], once);
        }
      }
    }
    // end mark, or wait for the copies in flight (those that a computing warp
    // still waits for need no wait here)
    if (!idle) {
      const int st = it % C::kStages;
      if (warp_wait(&empty[st], ((it / C::kStages) & 1) ^ 1, p)) {
        if (lead && lane == 0) desc[st].flags = kEnd;
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        if (!tma || lead) mbar_arrive(&full[st]);
      } else {
        late = true;
        for (int i = max(0, it - C::kStages); tma && i < it; ++i)
          mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, kDrainNs);
      }
    }
    copied = it;
    asm volatile("cp.async.wait_all;" ::: "memory");
    // an answer that nobody waited for (only after a wait ran out)
    if (answer_due) mbar_wait_bounded(&asked_full, answers & 1, kDrainNs);
    if (late) atomicMax(&trouble, 3);
  } else {
    // ------------------------------------------------------------ compute --
    const int row = lane >> 2, qd = lane & 3;
    const int mj = lane >> 3, mi = lane & 7;
    // ldmatrix row addresses: matrix mj, row mi
    const int tok0 = warp * 16 * C::kTiles;
    const uint32_t k_off = (tok0 + (mj & 1) * 8 + mi) * 128 + (((mj >> 1) ^ mi) << 4);
    const uint32_t v_off = C::kV + (tok0 + (mj >> 1) * 8 + mi) * 128 + (((mj & 1) ^ mi) << 4);
    const uint32_t q_off = mi * C::kQRow + mj * 16;               // two k-steps per load
    const uint32_t smb = smem_u32(sm);
    uint32_t qf[NT][D / 16][2];
    float o[NT][D / 16][4];
    float m[NT][2], l[NT][2];
    int meets = 0;
    bool dead = false;
    for (int it = 0; !dead; ++it) {
      const int st = it % C::kStages;
      if (!warp_wait(&full[st], (it / C::kStages) & 1, p)) { dead = true; break; }
      const BlockDesc b = desc[st];
      if (b.flags & kEnd) break;
      const uint32_t base = smb + st * C::kStage;
      if (b.flags & kFirst) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t r[4];
            ldsm4(smb + C::kStages * C::kStage + st * C::kQStage + t * 8 * C::kQRow + q_off + kk * 64,
                  r);
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
      const int nt = b.ntok - tok0;            // this warp's tokens
      if (nt > 0) {
        // the fragments of all K tiles, then of all V tiles, in batches: one is
        // loaded ahead of the products that use it
        constexpr int TT = C::kTiles, B = C::kBatch, KB = D / 16 / B, NB = TT * KB;
        constexpr int PP = std::is_same<Th, __half>::value ? 2 : 3;
        uint32_t fr[2][B][4];
        auto load = [&](int i) {                   // batch i of 2 NB
          const int tt = i / KB % TT, kb = i % KB;
          const uint32_t at = base + tt * 16 * 128;
#pragma unroll
          for (int e = 0; e < B; ++e) {            // 16 dims: two 16-byte units of a row
            const int kk = kb * B + e;
            const uint32_t unit = (uint32_t)(kk & 3) << 5, chunk = kk / 4 * C::kChunk;
            if (i < NB) ldsm4(((at + k_off) ^ unit) + chunk, fr[i & 1][e]);
            else ldsm4_t(((at + v_off) ^ unit) + chunk, fr[i & 1][e]);
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
        uint32_t part[PP][TT][NT][2];              // P's 16-bit parts, high to low
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
          const bool rise = (h0 < p.G && top[0] > m[t][0] + kTop) ||
                            (h0 + 1 < p.G && top[1] > m[t][1] + kTop);
          if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mb = top[e];
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 4));
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
              mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
              mb = fmaxf(mb - kLift, m[t][e]);
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
          // a reference of -inf (no finite score yet) must not meet itself
          const float ma = m[t][0] == -INFINITY ? 0.f : m[t][0];
          const float mb = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) {
            float p0 = ex2(x[tt][t][0] - ma), p1 = ex2(x[tt][t][1] - mb);
            float p2 = ex2(x[tt][t][2] - ma), p3 = ex2(x[tt][t][3] - mb);
            l[t][0] += p0 + p2;
            l[t][1] += p1 + p3;
#pragma unroll
            for (int i = 0; i < PP; ++i) {
              part[i][tt][t][0] = transpose8x8(take2(p0, p1, Th()));
              part[i][tt][t][1] = transpose8x8(take2(p2, p3, Th()));
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int tt = i / KB, vb = i % KB;
          if (i + 1 < NB) load(NB + i + 1);
          if (nt < 16 * TT) {
            // what lies behind the last row must not meet a weight of 0: it may be the
            // rest of a page, or of an earlier block, and hold anything
            const int t0 = 16 * tt + 2 * qd;
            const uint32_t keep0 = (t0 < nt ? 0xffffu : 0u) | (t0 + 1 < nt ? 0xffff0000u : 0u);
            const uint32_t keep1 = (t0 + 8 < nt ? 0xffffu : 0u) | (t0 + 9 < nt ? 0xffff0000u : 0u);
#pragma unroll
            for (int e = 0; e < B; ++e) {
              fr[(NB + i) & 1][e][0] &= keep0;
              fr[(NB + i) & 1][e][1] &= keep0;
              fr[(NB + i) & 1][e][2] &= keep1;
              fr[(NB + i) & 1][e][3] &= keep1;
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int part_i = 0; part_i < PP; ++part_i) {
              if (part_i == 2 && p.a.o_dtype != GDN_F32) break;
#pragma unroll
              for (int e = 0; e < B; ++e)
                mma16816<Th>(o[t][vb * B + e], fr[(NB + i) & 1][e], part[part_i][tt][t][0],
                             part[part_i][tt][t][1]);
            }
          }
        }
      }
      if (b.flags & kLast) {
        // the four warps' pieces meet over this block's K and V rows
        uint8_t* stage = sm + st * C::kStage;
        float* mine = reinterpret_cast<float*>(stage) + warp * C::kHeads * C::kPad;
        mbar_arrive(&meet);
        if (!warp_wait(&meet, meets & 1, p)) { dead = true; break; }
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
        if (!warp_wait(&meet, meets & 1, p)) { dead = true; break; }
        ++meets;
        const float* all = reinterpret_cast<const float*>(stage);
        int bad = 0;
#pragma unroll
        for (int w = 0; w < C::kPWarps; ++w) bad |= wrong_page[st][w];
        for (int i = tid; i < p.G * (D / 4); i += 32 * kCWarps) {
          const int h = i / (D / 4), d = 4 * (i % (D / 4));
          const int hq = b.g * p.G + h;
          const Gate<4> gate = load_gate<4>(a, b.n, hq, d);
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
          if (b.piece < 0) {
            const float inv = 1.f / L;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= inv;
            put_out<4>(a, (int64_t)b.n * a.Hq + hq, d, gate, y);
            if (a.lse && d == 0) a.lse[(int64_t)b.n * a.Hq + hq] = (M + log2f(L)) * kLn2;
          } else {
            const int64_t at = ((int64_t)b.range * 2 + b.piece) * p.G + h;
            *reinterpret_cast<float4*>(p.po + at * D + d) = make_float4(y[0], y[1], y[2], y[3]);
            if (d == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(M, L);
          }
        }
        fence_proxy_async_smem();              // written here before the next copies land
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (dead) atomicMax(&trouble, 3);           // a wait ran out: more than bad input
  }
  __syncthreads();
  // The join takes its place on the chip as CTAs end. It counts on this standing behind
  // every thread's wait_for_previous(), and any warp's call would count for the CTA: ahead
  // of the barrier, where copying warps without work made it at the start of the CTA,
  // the join's blocks came in beside the running ones (up to 1 us more).
  let_next_start();
  // nor may copies be in flight when the CTA ends that computing warps gave up waiting for
  if (trouble == 3 && p.box)
    for (int i = max(0, copied - C::kStages); i < copied; ++i)
      mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, kDrainNs);
  if (tid == 0) p.flag[blockIdx.x] = trouble == 3 ? 1 : trouble;
}

// Joins the pieces of sequences (and key-value heads) that start in one range
// and end in a later one; also sums up what the CTAs met. A warp takes one
// range and head; where a sequence has many pieces (a long one, alone), the
// block's warps share them.
// Where a wait ran out, a range may have no entry of this call (the CTA that was to
// write it gave up, or was taken over by one that did) and its place hold anything:
// then no entry is followed, and every row with tokens becomes NaN. Every block reads
// all flags for that, beside its entries (0.05 us; as a piece of code of its own behind
// a loop over the flags 0.3 us, the code being cold each time).
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps, kFewPieces = 8;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p, int ranges) {
  constexpr int V = D == 64 ? 2 : 4, K = D / 32 / V;       // a lane's K vectors of V floats
  __shared__ float acc[kJoinWarps][D];
  __shared__ int4 entry[kJoinWarps];
  const PagedDecodeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = blockIdx.x * kJoinWarps, h = blockIdx.y;
  const int4 none = make_int4(0, 0, 0, 0);
  const int c = c0 + warp;
  int4 mine;
  // First the rows of sequences without a token, or with a length out of range: nothing
  // of the split kernel's is needed for them. This stands ahead of the wait because the
  // split kernel lets the join start only after its own: what came before both is done,
  // and read from L2, where it is (a line of this SM's L1 may be older). Once more for
  // all others where a wait ran out.
  for (bool gave_up = false;; gave_up = true) {
    for (int n0 = blockIdx.x; n0 < a.N; n0 += 32 * gridDim.x) {   // 32 lengths at a time
      int len = 1;
      const int at = n0 + lane * gridDim.x;
      if (at < a.N)
        asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(len) : "l"(a.kv_lens + at)
                     : "memory");
      const bool ok = len_ok(a, len);
      uint32_t todo = __ballot_sync(0xffffffffu, at < a.N && (ok && len > 0) == gave_up);
      for (; todo; todo &= todo - 1) {
        const int k = __ffs(todo) - 1, n = n0 + k * gridDim.x;
        const bool nan = gave_up || !__shfl_sync(0xffffffffu, ok, k);
        for (int i = tid; i < a.Hkv * (D / 4); i += kJoinThreads) {
          const int hq = i / (D / 4) * p.G + h, d = 4 * (i % (D / 4));
          const float v = nan ? __int_as_float(0x7fc00000) : 0.f;
          float y[4] = {v, v, v, v};
          put_out<4>(a, (int64_t)n * a.Hq + hq, d, load_gate<4>(a, n, hq, d), y);
          if (a.lse && d == 0) a.lse[(int64_t)n * a.Hq + hq] = nan ? v : -INFINITY;
        }
      }
    }
    if (gave_up) return;
    wait_for_previous();
    let_next_start();
    mine = c < ranges ? p.join[c] : none;
    constexpr int kFlags = (kMaxRanges + kJoinThreads - 1) / kJoinThreads;
    int f = 0;
#pragma unroll
    for (int i = 0; i < kFlags; ++i)
      f |= tid + i * kJoinThreads < ranges ? p.flag[tid + i * kJoinThreads] : 0;
    const bool timeout = __syncthreads_or(f & 1);
    if (blockIdx.x == 0 && h == 0) {
      const int wrong = __syncthreads_or(f & 2);
      if (tid == 0) *p.status = timeout ? 1 : (wrong ? 2 : 0);
    }
    if (!timeout) break;
  }
  // one warp's sum over pieces first, first + step, ...; returns the max and sum
  // over all pieces. Loads go out several at a time.
  auto gather = [&](int c, const int4& j, int first, int step, float (&y)[K][V]) -> float2 {
    const int pieces = j.z - c + 1;
    auto at = [&](int i) { return ((int64_t)(c + i) * 2 + (i == 0)) * p.G + h; };
    auto weight = [](float m, float M) { return m == -INFINITY ? 1.f : ex2(m - M); };
    float M = -INFINITY, L = 0.f;
    for (int i0 = lane; i0 < pieces; i0 += 128) {
      float2 ml[4];
      float top = M;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ml[e] = i0 + 32 * e < pieces ? *reinterpret_cast<const float2*>(p.ml + at(i0 + 32 * e) * 2)
                                     : make_float2(-INFINITY, 0.f);
        top = fmaxf(top, ml[e].x);
      }
      L *= weight(M, top);
#pragma unroll
      for (int e = 0; e < 4; ++e) L += weight(ml[e].x, top) * ml[e].y;
      M = top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
      const float top = fmaxf(M, m2);
      const float a1 = weight(M, top) * L, a2 = weight(m2, top) * l2;
      L = lane & o ? a2 + a1 : a1 + a2;            // the same order in both lanes
      M = top;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) y[k][e] = 0.f;
    constexpr int R = kFewPieces;
    for (int i0 = first; i0 < pieces; i0 += R * step) {
      float m[R], v[R][K][V];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool live = i0 + r * step < pieces;
        const int64_t x = at(live ? i0 + r * step : i0);
        m[r] = live ? p.ml[x * 2] : INFINITY;
        const float* src = p.po + x * D + lane * V;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if constexpr (V == 4)
            *reinterpret_cast<float4*>(v[r][k]) = *reinterpret_cast<const float4*>(src + k * 32 * V);
          else
            *reinterpret_cast<float2*>(v[r][k]) = *reinterpret_cast<const float2*>(src + k * 32 * V);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (i0 + r * step < pieces) {
          const float f = weight(m[r], M);
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) y[k][e] += f * v[r][k][e];
        }
      }
    }
    return make_float2(M, L);
  };
  struct Gates { Gate<V> g[K]; };
  auto gates = [&](const int4& j) {
    Gates r;
#pragma unroll
    for (int k = 0; k < K; ++k) r.g[k] = load_gate<V>(a, j.x, j.y * p.G + h, (k * 32 + lane) * V);
    return r;
  };
  auto finish = [&](const int4& j, float2 ml, const Gates& g, float (&y)[K][V]) {
    const int hq = j.y * p.G + h;
    const int64_t row = (int64_t)j.x * a.Hq + hq;
    const float inv = 1.f / ml.y;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < V; ++e) y[k][e] *= inv;
      put_out<V>(a, row, (k * 32 + lane) * V, g.g[k], y[k]);
    }
    if (a.lse && lane == 0) a.lse[row] = (ml.x + log2f(ml.y)) * kLn2;
  };
  if (lane == 0) entry[warp] = mine;
  const bool many = mine.w && mine.z - c + 1 > kFewPieces;
  float y[K][V];
  if (mine.w && !many) {
    const Gates g = gates(mine);
    const float2 ml = gather(c, mine, 0, 1, y);
    finish(mine, ml, g, y);
  }
  if (!__syncthreads_or(many)) return;
  for (int w = 0; w < kJoinWarps && c0 + w < ranges; ++w) {
    const int4 j = entry[w];
    if (!j.w || j.z - (c0 + w) + 1 <= kFewPieces) continue;
    const Gates g = gates(j);
    const float2 ml = gather(c0 + w, j, warp, kJoinWarps, y);
    __syncthreads();                           // the last turn's sums are read
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[warp][(k * 32 + lane) * V + e] = y[k][e];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
          for (int i = 1; i < kJoinWarps; ++i) y[k][e] += acc[i][(k * 32 + lane) * V + e];
      finish(j, ml, g, y);
    }
  }
}

// most ranges of a launch: D = 64 has two CTAs per SM
constexpr int max_ranges(int D) { return D == 64 ? kMaxRanges : kMaxRanges / 2; }
constexpr size_t kHeadBytes = 256 + kMaxRanges * 4 + kMaxRanges * 16;

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = found.load(std::memory_order_relaxed);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* ptr = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    found.store(fn, std::memory_order_relaxed);
  }
  return fn;
}
// A cache as [page][token][head][D] or [page][head][token][D], the smaller stride
// inside; boxes of p.box tokens of one head by 64 dims. False where a map cannot
// say it: each stride has to be a multiple of the one inside it, below 2^40 bytes.
bool make_map(CUtensorMap* map, const void* base, const PageStrides& s, const PagedParams& p,
              bool* token_first) {
  auto fn = map_encoder();
  if (!fn) return false;
  const int page_size = p.a.page_size, heads = p.a.Hkv;
  *token_first = heads == 1 || (page_size > 1 && s.token < s.head);
  const cuuint64_t size[2] = {(cuuint64_t)(*token_first ? page_size : heads),
                              (cuuint64_t)(*token_first ? heads : page_size)};
  cuuint64_t strides[3] = {(cuuint64_t)(*token_first ? s.token : s.head) * 2,
                           (cuuint64_t)(*token_first ? s.head : s.token) * 2,
                           (cuuint64_t)s.page * 2};
  if (size[0] == 1) strides[0] = (cuuint64_t)p.a.D * 2;        // never used
  if (size[1] == 1) strides[1] = strides[0] * size[0];
  if (p.a.num_pages == 1) strides[2] = strides[1] * size[1];
  if (strides[1] % strides[0] || strides[2] % strides[1] || strides[2] >> 40) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)p.a.D, size[0], size[1], (cuuint64_t)p.a.num_pages};
  const cuuint32_t rows = (cuuint32_t)p.box;
  const cuuint32_t box[4] = {64, *token_first ? rows : 1, *token_first ? 1 : rows, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(map,
            p.a.kv_dtype == GDN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
            4, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, class Th>
cudaError_t launch_split(PagedParams p, int sms) {
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
  p.base = min(sms * C::kCtasPerSm, max_ranges(D) / kPhases);
  // ranges to take over only where the tables have room for enough units (the lengths
  // are not known here: under a table far wider than they are the CTAs past the base find
  // one phase and have to be cancelled; 8 short sequences with rows for 131072 tokens
  // 11.8 us, for 300 10.9)
  const int64_t cap = (int64_t)p.a.max_pages * p.a.page_size;
  const int64_t most = (cap + C::kTok - 1) / C::kTok * p.a.N * p.a.Hkv;
  const int grid = most >= kStealUnits * (int64_t)p.base ? kPhases * p.base : p.base;
  // copies by TMA where the page size has a factor of 8 rows, 16 at D = 256. Against
  // cp.async, one after the other on one B200 before the power cap bit: 256 x 4097
  // tokens, D = 256, pages of 64: 616 us, 666; 64 x 4097, pages of
  // 16: D = 256 168, 180, D = 128 166, 169, D = 64 182, 193; pages of 8: 191, 180;
  // 171, 169; 175, 192
  CUtensorMap k_map{}, v_map{};
  p.box = p.a.page_size & -p.a.page_size;
  if (p.box > C::kTok) p.box = C::kTok;
  if (p.box < (D == 256 ? 16 : 8) || !make_map(&k_map, p.a.k_cache, p.a.ks, p, &p.k_token_first) ||
      !make_map(&v_map, p.a.v_cache, p.a.vs, p, &p.v_token_first))
    p.box = 0;
  // a warp for every eight copies of each side
  p.copy_warps = C::kPWarps;
  if (p.box) {
    const int copies = C::kTok / p.box * (D / 64);
    p.copy_warps = 2 * max(1, min(copies / 8, C::kPWarps / 2));
  }
  e = launch_early(paged_split_kernel<D, NT, Th>, dim3((unsigned)grid), C::kThreads, C::kSmem,
                   p.a.stream, p, k_map, v_map);
  if (e != cudaSuccess) return e;
  // the join's CTAs come in while the split's last ones end, and wait for them
  return launch_early(paged_join_kernel<D>,
                      dim3((unsigned)((grid + kJoinWarps - 1) / kJoinWarps), (unsigned)p.G),
                      kJoinThreads, 0, p.a.stream, p, grid);
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
  return kHeadBytes + (size_t)max_ranges(D) * 2 * group * (D + 2) * 4;
}

cudaError_t launch_paged_decode(const PagedDecodeArgs& a) {
  if (a.N == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PagedParams p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.limit_ns = wait_limit_ns();
  p.poll = p.limit_ns < kSuspendNs;
  p.status = reinterpret_cast<int*>(ws);
  p.flag = reinterpret_cast<int*>(ws + 256);
  p.join = reinterpret_cast<int4*>(ws + 256 + kMaxRanges * 4);
  p.po = reinterpret_cast<float*>(ws + kHeadBytes);
  p.ml = p.po + (size_t)max_ranges(a.D) * 2 * p.G * a.D;
  return a.kv_dtype == GDN_F16 ? launch_dim<__half>(p, sms) : launch_dim<__nv_bfloat16>(p, sms);
}

}  // namespace gdn
