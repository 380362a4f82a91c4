// Page plan of a paged key-value cache: request lengths go in, block-table
// entries, the free stack, a slot and a position for every new token come out,
// in one launch and without a host round trip.
//
// Requests move from lens[n] to want[n] tokens. With held = ceil(lens / page)
// and goal = ceil(want / page), a shrinking request returns its table entries
// goal..held-1, in request order, on top of the free stack; growing requests
// then take pages from the stack's top, in request order. Growth is granted to
// the longest prefix of the growing requests whose pages and tokens fit, which
// two running sums decide: both are non-decreasing, so "fits" turns false once.
//
// Every CTA makes the three running sums (tokens, pages taken, pages returned)
// over all requests for itself in shared memory and then works on its share of
// the pages and tokens by searching them: no CTA waits for another, and nothing
// is kept in a workspace. That needs the inputs to stay as they are during the
// launch: new lengths and the new count go to their own arrays; the stack below
// the old count is only read, above it only written; table rows of shrinking
// requests are only read, of growing ones only written past their held pages.
// So a call repeated on the same inputs gives the same outputs.
//
// Latency bounds it: 64 requests 6.8 us, 509 with 8192 tokens 9.4, 4096 with room
// for 262144 tokens 13.0 (2.2 MB; each CTA's sums are most of it), of which a launch
// is 2. Requests read once instead of in each pass, divisions by multiplication
// and a CTA sized to the step took it there from 8.6, 11.6 and 17.6.
//
// Two kinds of step are far from that. The grid goes by the token budget alone: 25
// requests of 16384 tokens that end (25600 pages) take 112 us with room for 512 tokens,
// 6.4 with room for 65536. And a token's request is searched once per four tokens and
// then walked to, past every request that does not grow: of 16384 requests two growing
// ones at the ends take 482 us, 64 spread ones 90, all of them 59 (of 1024: 31, 8, 5.6).
#include "gdn_common.cuh"
#include "launch.h"
#include "pdl.cuh"

namespace gdn {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kKeep = 4;          // requests a thread keeps in registers

struct Sums { uint32_t tok, take, back; };

struct PlanShared {
  Sums warp[kMaxThreads / 32];
  Sums total, grant;      // grant: sums over the granted requests
  uint32_t refused;
};

// Saturating running sums: past the limits only "does not fit" is of interest.
struct Limits { uint32_t tok, take; };
__device__ __forceinline__ Sums add(const Sums& a, const Sums& b, const Limits& lim) {
  return Sums{min(a.tok + b.tok, lim.tok), min(a.take + b.take, lim.take), a.back + b.back};
}
__device__ __forceinline__ Sums shfl_up(const Sums& s, int o) {
  return Sums{__shfl_up_sync(0xffffffffu, s.tok, o), __shfl_up_sync(0xffffffffu, s.take, o),
              __shfl_up_sync(0xffffffffu, s.back, o)};
}

// Largest i in [0, n) with a[i] <= x (a[0] = 0, non-decreasing).
__device__ __forceinline__ int last_le(const uint32_t* a, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

struct PlanParams {
  PagePlanArgs a;
  FastDiv page;
};

// A request: its lengths, and what it asks of the running sums.
struct Request {
  int len, want;
  Sums s;
  __device__ bool grow() const { return s.tok != 0; }
  __device__ bool shrink() const { return valid && want < len; }
  bool valid;
};
__device__ __forceinline__ Request request(const PlanParams& p, int n, const Limits& lim) {
  Request r{p.a.lens[n], p.a.want[n], Sums{0u, 0u, 0u}, false};
  const int64_t cap = (int64_t)p.a.max_pages * p.a.page_size;
  r.valid = r.len >= 0 && r.want >= 0 && r.len <= cap && r.want <= cap;
  if (r.valid) {
    const int pages = p.page.up(r.want) - p.page.up(r.len);
    if (r.want > r.len) {
      r.s.tok = min((uint32_t)(r.want - r.len), lim.tok);
      r.s.take = min((uint32_t)pages, lim.take);
    } else {
      r.s.back = (uint32_t)-pages;
    }
  }
  return r;
}

// KEEP: at most kKeep requests per thread, read once and kept.
template <bool KEEP>
__global__ void __launch_bounds__(kMaxThreads) page_plan_kernel(const PlanParams pp) {
  extern __shared__ uint32_t sums[];            // cu | take | back, N + 1 each
  __shared__ PlanShared sh;
  const PagePlanArgs& p = pp.a;
  uint32_t* cu = sums;
  uint32_t* take = sums + (p.N + 1);
  uint32_t* back = take + (p.N + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const Limits lim{(uint32_t)p.token_capacity + 1u, (uint32_t)p.num_pages + 1u};
  const bool writer = blockIdx.x == 0;
  if (tid == 0) sh.refused = 0;
  let_next_start();
  wait_for_previous();

  // running sums: a run of requests per thread, then over the threads
  const int per = (p.N + threads - 1) / threads;
  const int n0 = min(tid * per, p.N), n1 = min(n0 + per, p.N);
  Request kept[KEEP ? kKeep : 1];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (n0 + i < n1) kept[i] = request(pp, n0 + i, lim);
  }
  auto each = [&](auto&& body) {
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (n0 + i < n1) body(n0 + i, kept[i]);
    } else {
      for (int n = n0; n < n1; ++n) body(n, request(pp, n, lim));
    }
  };
  const uint32_t count = (uint32_t)min(max(p.free_count[0], 0), p.num_pages);
  Sums mine{0u, 0u, 0u};
  each([&](int, const Request& r) { mine = add(mine, r.s, lim); });
  Sums incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v = shfl_up(incl, o);
    if (lane >= o) incl = add(v, incl, lim);
  }
  if (lane == 31) sh.warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    Sums w = lane < threads / 32 ? sh.warp[lane] : Sums{0u, 0u, 0u};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums v = shfl_up(w, o);
      if (lane >= o) w = add(v, w, lim);
    }
    sh.warp[lane] = w;
    if (lane == 31) { sh.total = w; sh.grant = w; }
  }
  __syncthreads();
  Sums run = shfl_up(incl, 1);                  // exclusive within the warp
  if (lane == 0) run = Sums{0u, 0u, 0u};
  if (warp > 0) run = add(sh.warp[warp - 1], run, lim);

  const uint32_t back_all = min(sh.total.back, (uint32_t)p.num_pages - count);
  const uint32_t avail = count + back_all;      // entries of the stack after the returns
  auto fits = [&](const Sums& s) {
    return s.take <= avail && s.tok <= (uint32_t)p.token_capacity;
  };
  // the request at which "fits" turns false (at most one) gives the granted sums
  if (!fits(sh.total)) {
    Sums r = run;
    each([&](int, const Request& q) {
      const Sums next = add(r, q.s, lim);
      if (fits(r) && !fits(next)) { sh.grant.tok = r.tok; sh.grant.take = r.take; }
      r = next;
    });
    __syncthreads();
  }
  const uint32_t tok_all = sh.grant.tok, take_all = sh.grant.take;
  int refused = 0;
  each([&](int n, const Request& q) {
    const Sums next = add(run, q.s, lim);
    const bool before = fits(run);
    cu[n] = before ? run.tok : tok_all;
    take[n] = before ? run.take : take_all;
    back[n] = run.back;
    if (writer) {
      const bool ok = q.shrink() || (q.grow() && fits(next));
      p.new_lens[n] = ok ? q.want : q.len;
      p.cu_new[n] = (int)cu[n];
      refused += q.want != q.len && !ok;
    }
    run = next;
  });
  if (refused) atomicAdd(&sh.refused, (uint32_t)refused);
  if (tid == 0) { cu[p.N] = tok_all; take[p.N] = take_all; back[p.N] = sh.total.back; }
  __syncthreads();
  if (writer && tid == 0) {
    p.cu_new[p.N] = (int)tok_all;
    p.new_count[0] = (int)(avail - take_all);
    if (p.info) {
      p.info[0] = (int)tok_all;
      p.info[1] = (int)take_all;
      p.info[2] = (int)back_all;
      p.info[3] = (int)sh.refused;
    }
  }

  // entry v of the stack after the returns
  auto entry = [&](uint32_t v) -> int {
    if (v < count) return p.free_pages[v];
    const uint32_t w = v - count;
    const int m = last_le(back, p.N, w);
    const int goal = pp.page.up(p.want[m]);
    return p.table[(int64_t)m * p.table_row_stride + goal + (int)(w - back[m])];
  };
  const uint32_t first = blockIdx.x * threads + tid, step = gridDim.x * threads;
  // where taken page i goes
  auto taken_at = [&](uint32_t i) -> int64_t {
    const int m = last_le(take, p.N, i);
    return (int64_t)m * p.table_row_stride + pp.page.up(p.lens[m]) + (int)(i - take[m]);
  };
  // A thread's first taken and first returned page are read before its tokens and
  // written after them, so that the three reads' latencies pass together.
  const uint32_t put_end = avail - take_all;     // returned pages stay at count .. put_end - 1
  const bool take_one = first < take_all, put_one = count + first < put_end;
  const int64_t take_to = take_one ? taken_at(first) : 0;
  const int take_page = take_one ? entry(avail - 1 - first) : 0;
  const int put_page = put_one ? entry(count + first) : 0;

  // four tokens per thread and round: one search, then forward
  for (int64_t t0 = 4 * (int64_t)first; t0 < p.token_capacity; t0 += 4 * (int64_t)step) {
    int slot[4], pos[4];
    int m = 0, last_m = -1, last_j = -1, page = -1;
    if (t0 < tok_all) m = last_le(cu, p.N, (uint32_t)t0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t t = (uint32_t)t0 + e;
      slot[e] = -1;
      pos[e] = 0;
      if (t < tok_all) {
        while (t >= cu[m + 1]) ++m;             // ends: cu[N] = tok_all > t
        const int len = p.lens[m];
        pos[e] = len + (int)(t - cu[m]);
        const int j = pp.page(pos[e]);
        if (m != last_m || j != last_j) {
          const int held = pp.page.up(len);
          page = j < held ? p.table[(int64_t)m * p.table_row_stride + j]
                          : entry(avail - 1 - (take[m] + (uint32_t)(j - held)));
          last_m = m;
          last_j = j;
        }
        if (page >= 0 && page < p.num_pages)
          slot[e] = page * p.page_size + (pos[e] - j * p.page_size);
      }
    }
    if (t0 + 4 <= p.token_capacity) {
      *reinterpret_cast<int4*>(p.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (p.positions)
        *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int e = 0; e < (int)(p.token_capacity - t0); ++e) {
        p.slot_map[t0 + e] = slot[e];
        if (p.positions) p.positions[t0 + e] = pos[e];
      }
    }
  }
  if (take_one) p.table[take_to] = take_page;
  if (put_one) p.free_pages[count + first] = put_page;
  for (uint32_t i = first + step; i < take_all; i += step)
    p.table[taken_at(i)] = entry(avail - 1 - i);
  for (uint32_t v = count + first + step; v < put_end; v += step) p.free_pages[v] = entry(v);
}

}  // namespace

cudaError_t launch_page_plan(const PagePlanArgs& a) {
  const size_t smem = 3 * sizeof(uint32_t) * ((size_t)a.N + 1);
  const PlanParams p{a, FastDiv(a.page_size)};
  auto kernel = a.N <= kKeep * kMaxThreads ? page_plan_kernel<true> : page_plan_kernel<false>;
  if (smem > 32 * 1024) {
    // always the largest size, so that concurrent calls do not lower each other's limit
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)(3 * sizeof(uint32_t) * (kPlanMaxRequests + 1)));
    if (e != cudaSuccess) return e;
  }
  // threads for a request and four tokens each, in one CTA where that goes; then
  // one CTA per 4096 tokens of the budget, up to one per SM
  const int64_t work = a.token_capacity / 4 > a.N ? a.token_capacity / 4 : a.N;
  const int threads = work <= 128 ? 128 : (work <= 512 ? 512 : kMaxThreads);
  const int64_t want = (a.token_capacity + 4 * threads - 1) / (4 * threads);
  const unsigned grid = (unsigned)(want < 1 ? 1 : (want > 148 ? 148 : want));
  return launch_early(kernel, dim3(grid), (unsigned)threads, smem, a.stream, p);
}

}  // namespace gdn
