// Eviction from a paged cache by accumulated attention weight.
//
// For a stream (sequence b, KV head h) of n tokens and a budget of m < n: the
// protected tokens and, of the others, those with the largest accumulated
// weight are kept, ties to the lower slot.  Kept tokens at slots >= m move
// into the freed slots < m: sources and targets are disjoint, so the move
// needs no order and happens in place, and only what has to move does.
//
// select: exact radix selection of the m-th largest 31-bit key (weights are
// not negative, so their bits are ordered; protected tokens have the largest
// key), then one ordered pass that ranks freed slots and movers by per-warp
// counts.  move: rows and bookkeeping, wide.
//
// What bounds it: select reads 8 bytes a token once from DRAM and is then
// bound by the latency of its few cluster-wide steps; move by DRAM, 4 rows of
// traffic per moved token.  Measured, both together: 64 streams of 4097 to 4096
// 9.4 us; 32 streams of 32768 to 2048 (fp16 rows of 128) 30.7 us, of which 9 are
// select's 18 thousand cycles; 8 streams of 1048576 to 8192 62.8 us, the pass over
// 67 MB by 64 SMs 15 us of them.
#include <cooperative_groups.h>

#include "decode_common.cuh"
#include "paged_internal.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace mkv {
namespace {

constexpr int ET = 1024, EW = ET / 32;
constexpr int E_BINS = 2048;
constexpr int E_SHORT = 16 * ET;          // slots of a slice whose keys stay in registers
constexpr uint32_t KEY_SAFE = 0x7fffffffu;

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  const int n = p.lens[b];
  return n < 0 ? 0 : min(n, p.limit);
}

// Sum over the block of v before this thread (exclusive); total in *all.
__device__ __forceinline__ int block_prefix(int v, int* ws, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) ws[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int u = ws[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(~0u, u, o);
      if (lane >= o) u += t;
    }
    ws[lane] = u;
  }
  __syncthreads();
  *all = ws[EW - 1];
  return inc - v + (warp ? ws[warp - 1] : 0);
}

// What both selection kernels know of their stream and slice.
struct Slice {
  const float* acc;
  const int32_t* pos;
  int32_t *src, *movers, *holes;
  int64_t from;                           // positions from here on are protected
  int n, m, sink;
  int sl, s0, s1, wl, w0, w1;             // slots of a CTA; this CTA's; of a warp; this warp's
};

__device__ __forceinline__ uint32_t form_key(const Slice& s, float a, int q) {
  if (q < s.sink || q >= s.from) return KEY_SAFE;
  return a > 0.f ? __float_as_uint(a) : 0u;
}

template <int R>
__device__ __forceinline__ void cluster_barrier() {
  if constexpr (R > 1) cg::this_cluster().sync(); else __syncthreads();
}

// Fills `s`; false where nothing is to be evicted (then src is written).
template <int R>
__device__ __forceinline__ bool slice_of(const EvictParams& p, int rank, Slice& s) {
  const int64_t stream = blockIdx.x / R;
  const int b = (int)(stream / p.H), h = (int)(stream - (int64_t)b * p.H);
  s.n = evict_len(p, b);
  s.m = p.budget;
  s.src = p.src + stream * s.m;
  if (h == 0 && rank == 0 && threadIdx.x == 0 && p.status && p.lens[b] != s.n) atomicOr(p.status, DEV_ERR_CHECK);
  if (s.n <= s.m) {
    for (int64_t i = rank * ET + threadIdx.x; i < s.m; i += (int64_t)R * ET) s.src[i] = i < s.n ? (int)i : -1;
    return false;
  }
  s.acc = p.acc + stream * p.meta_stride;
  s.pos = p.pos + stream * p.meta_stride;
  s.movers = p.lists + stream * 2 * s.m;         // s.m < s.n <= p.limit here
  s.holes = s.movers + s.m;
  s.sink = p.sink;
  s.from = (int64_t)p.next_pos[b] - p.recent;
  s.sl = ((s.n + R - 1) / R + ET - 1) / ET * ET;
  s.wl = s.sl / EW;
  s.s0 = min(s.n, rank * s.sl);
  s.s1 = min(s.n, s.s0 + s.sl);
  s.w0 = min(s.s1, s.s0 + ((int)threadIdx.x >> 5) * s.wl);
  s.w1 = min(s.s1, s.w0 + s.wl);
  return true;
}

// Adds this CTA's histogram into every rank's `total` (few of its bins are in
// use: a push of those costs less than every rank's reading of R whole
// histograms, 10 against 2 thousand cycles for 2048 bins of 8 ranks), then
// finds the bin of the `need`-th largest key: pick = {bin, keys in bins above,
// keys in it}.  Returns the keys in all.  `total` must be zero in every rank.
template <int R>
__device__ __forceinline__ int pick_bin(int* hist, int* total, int bins, int need, int* ws, int* pick) {
  constexpr int MAXPER = E_BINS / ET;
  const int per = bins / ET;
  if constexpr (R > 1) {
    cg::cluster_group cl = cg::this_cluster();
    __syncthreads();
#pragma unroll
    for (int x = 0; x < MAXPER; ++x)
      if (x < per) {
        const int bin = x * ET + (int)threadIdx.x, v = hist[bin];
        if (v) {
#pragma unroll
          for (int q = 0; q < R; ++q) atomicAdd(cl.map_shared_rank(&total[bin], q), v);
        }
      }
    cl.sync();
  } else {
    __syncthreads();
    total = hist;
  }
  int mine[MAXPER] = {}, sum = 0;
#pragma unroll
  for (int x = 0; x < MAXPER; ++x)
    if (x < per) {
      mine[x] = total[bins - 1 - ((int)threadIdx.x * per + x)];   // from the top
      sum += mine[x];
    }
  int all;
  int before = block_prefix(sum, ws, &all);
#pragma unroll
  for (int x = 0; x < MAXPER; ++x)
    if (x < per) {
      if (before < need && before + mine[x] >= need) {
        pick[0] = bins - 1 - ((int)threadIdx.x * per + x);
        pick[1] = before;
        pick[2] = mine[x];
      }
      before += mine[x];
    }
  __syncthreads();
  return all;
}

// From every warp's counts (keys above the limit, and equal to it, below and
// from slot m): equal keys, movers and freed slots of all warps before this
// one, in slot order, and all movers.  Lane i takes warp i of every rank.
struct Ranks {
  int eq, movers, holes, all_movers;
};
template <int R>
__device__ __forceinline__ Ranks rank_warps(const Slice& s, int4* cnt, int need, int rank) {
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Ranks o = {0, 0, 0, 0};
  int4 e[R];
#pragma unroll
  for (int q = 0; q < R; ++q) e[q] = R > 1 ? *cl.map_shared_rank(&cnt[lane], q) : cnt[lane];
  int run_eq = 0, run_mv = 0, run_ho = 0;
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int eqs = e[q].z + e[q].w;
    int inc = eqs;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const int u = __shfl_up_sync(~0u, inc, o2);
      if (lane >= o2) inc += u;
    }
    const int eb = run_eq + inc - eqs;
    const int k0 = min(max(need - eb, 0), e[q].z), k1 = min(max(need - eb - e[q].z, 0), e[q].w);
    const int r0 = min(s.n, q * s.sl), r1 = min(s.n, r0 + s.sl);
    const int first = min(r1, r0 + lane * s.wl), last = min(r1, first + s.wl);
    const int mv = e[q].y + k1, ho = max(0, min(last, s.m) - first) - e[q].x - k0;
    int im = mv, ih = ho;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const int u = __shfl_up_sync(~0u, im, o2), v = __shfl_up_sync(~0u, ih, o2);
      if (lane >= o2) im += u, ih += v;
    }
    if (q == rank) {
      o.eq = __shfl_sync(~0u, eb, warp);
      o.movers = run_mv + __shfl_sync(~0u, im - mv, warp);
      o.holes = run_ho + __shfl_sync(~0u, ih - ho, warp);
    }
    run_eq += __shfl_sync(~0u, inc, 31);
    run_mv += __shfl_sync(~0u, im, 31);
    run_ho += __shfl_sync(~0u, ih, 31);
  }
  o.all_movers = run_mv;
  return o;
}

// Writes the movers and freed slots of 32 slots from t0 on, given as bit masks,
// into the lists.  The ranks are below m; the checks hold that too where
// another stream writes the weights meanwhile and passes see different keys.
__device__ __forceinline__ void list_word(const Slice& s, Ranks& k, int t0, unsigned mv, unsigned ho) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  const int im = k.movers + __popc(mv & below), ih = k.holes + __popc(ho & below);
  if ((mv >> lane & 1) && im >= 0 && im < s.m) s.movers[im] = t0 + lane;
  if ((ho >> lane & 1) && ih >= 0 && ih < s.m) s.holes[ih] = t0 + lane;
  k.movers += __popc(mv);
  k.holes += __popc(ho);
}

// The i-th freed slot receives the i-th mover.
template <int R>
__device__ __forceinline__ void fill_holes(const Slice& s, int all_movers, int rank) {
  cluster_barrier<R>();                   // lists are complete, and no rank's counts are read any more
  for (int i = rank * ET + threadIdx.x; i < min(all_movers, s.m); i += R * ET) {
    const int t = s.holes[i];
    if (t >= 0 && t < s.m) s.src[t] = s.movers[i];
  }
}

// ---------------------------------------------------------------------------
// select, short slices: every key stays in a register, slot w0 + 32 j + lane in
// register j, so that a ballot is 32 slots in order.  Each level has a
// histogram of its own: nothing that another rank still needs is written again.
//
// In the steady state few tokens leave (one a step): up to E_FEW of them are
// found one by one as the smallest (key, highest slot) instead, without any
// histogram, and every thread then knows them all (64 streams of 4097: 15 us a
// cold call, 21 through the histograms).
// grid: streams * R, cluster R; block 1024
// ---------------------------------------------------------------------------
constexpr int E_FEW = 4;
constexpr int E_HIST = E_BINS + 2 * (E_BINS / 2);   // three levels

template <int R, int KPT>
__global__ void __launch_bounds__(ET, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[E_HIST], total[R > 1 ? E_HIST : 1];
  __shared__ int ws[EW];
  __shared__ int4 cnt[EW];
  __shared__ int pick[3];
  __shared__ uint2 least[2][EW], leave[E_FEW], left[E_FEW];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = R > 1 ? (int)cl.block_rank() : 0;
  griddep_wait();
  griddep_launch();
  Slice s;
  if (!slice_of<R>(p, rank, s)) return;
  float a[KPT];
  int pos[KPT];
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int t = s.w0 + 32 * j + lane;
    if (t < s.w1) a[j] = s.acc[t], pos[j] = s.pos[t];
  }
  uint32_t key[KPT];
  auto form = [&](int j) {
    key[j] = s.w0 + 32 * j + lane < s.w1 ? form_key(s, a[j], pos[j]) : 0u;
  };
  if (s.n - s.m <= E_FEW) {
#pragma unroll
    for (int j = 0; j < KPT; ++j) form(j);
    // smallest key, of equal ones the highest slot: (key, ~slot) ascending
    const int few = s.n - s.m;
    unsigned gone = 0;                    // registers whose token leaves
    for (int e = 0; e < few; ++e) {
      uint32_t k = ~0u, inv = ~0u;        // ~slot
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const int t = s.w0 + 32 * j + lane;
        if (t < s.w1 && !(gone >> j & 1) && key[j] <= k) k = key[j], inv = ~(uint32_t)t;
      }
      const uint32_t wk = __reduce_min_sync(~0u, k);
      const uint32_t wi = __reduce_min_sync(~0u, k == wk ? inv : ~0u);
      if (lane == 0) least[e & 1][warp] = make_uint2(wk, wi);
      __syncthreads();
      const uint2 v = least[e & 1][lane];
      const uint32_t bk = __reduce_min_sync(~0u, v.x);
      const uint32_t bi = __reduce_min_sync(~0u, v.x == bk ? v.y : ~0u);
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (~(uint32_t)(s.w0 + 32 * j + lane) == bi) gone |= 1u << j;
      if (tid == 0) (R > 1 ? leave : left)[e] = make_uint2(bk, bi);
    }
    if constexpr (R > 1) {
      // of every rank's smallest, the smallest
      cl.sync();
      if (warp == 0) {
        uint2 v = make_uint2(~0u, ~0u);
        if (lane < R * E_FEW && lane % E_FEW < few) v = *cl.map_shared_rank(&leave[lane % E_FEW], lane / E_FEW);
        for (int e = 0; e < few; ++e) {
          const uint32_t k = __reduce_min_sync(~0u, v.x);
          const uint32_t i = __reduce_min_sync(~0u, v.x == k ? v.y : ~0u);
          if (lane == 0) left[e] = make_uint2(k, i);
          if (v.y == i) v = make_uint2(~0u, ~0u);
        }
      }
      cl.sync();                          // no rank's candidates are read any more
    } else {
      __syncthreads();
    }
    // the slots that leave, and the kept ones from slot m on, in order
    int out[E_FEW];
#pragma unroll
    for (int e = 0; e < E_FEW; ++e) out[e] = e < few ? (int)~left[e].y : 0x7fffffff;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int t = s.w0 + 32 * j + lane;
      if (t < s.w1 && t < s.m) {
        int from = t, place = 0;
        bool is_out = false;
#pragma unroll
        for (int e = 0; e < E_FEW; ++e) is_out |= out[e] == t, place += out[e] < t;
        if (is_out) {
          // the place-th of slots m .. n - 1 that stay
          int k = -1;
          for (from = s.m - 1; k < place && from < s.n - 1;) {
            ++from;
            bool stays = true;
#pragma unroll
            for (int e = 0; e < E_FEW; ++e) stays &= out[e] != from;
            k += stays;
          }
        }
        s.src[t] = from;
      }
    }
    return;
  }
  for (int i = tid; i < E_HIST; i += ET) {
    hist[i] = 0;
    if constexpr (R > 1) total[i] = 0;
  }
  if constexpr (R > 1) cl.barrier_arrive();   // totals are zero
  __syncthreads();
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    form(j);
    if (s.w0 + 32 * j + lane < s.w1) atomicAdd(&hist[key[j] >> 20], 1);
  }
  if constexpr (R > 1) cl.barrier_wait();
  // the m-th largest key, 11 + 10 + 10 bits at a time: keys > lim are kept, and
  // of those equal to lim the `need` with the lowest slots
  uint32_t lim = 0;
  int need = s.m;
#pragma unroll
  for (int level = 0; level < 3; ++level) {
    constexpr int kShift[3] = {20, 10, 0}, kBase[3] = {0, E_BINS, E_BINS + E_BINS / 2};
    const int shift = kShift[level];
    int* hl = hist + kBase[level];
    if (level > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (s.w0 + 32 * j + lane < s.w1 && (key[j] ^ lim) >> (shift + 10) == 0u)
          atomicAdd(&hl[(key[j] >> shift) & 1023], 1);
    }
    pick_bin<R>(hl, total + (R > 1 ? kBase[level] : 0), level == 0 ? E_BINS : E_BINS / 2, need, ws, pick);
    lim |= (uint32_t)pick[0] << shift;
    need -= pick[1];
    if (pick[2] == need) {                // the whole bin is kept: keys > lim - 1
      need = 0;
      break;
    }
  }
  const int64_t over = need == 0 ? (int64_t)lim - 1 : (int64_t)lim;
  {
    int c0 = 0, c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int t = s.w0 + 32 * j + lane;
      const int u = t < s.w1 && (int64_t)key[j] > over, e = t < s.w1 && need && key[j] == lim;
      if (t < s.m) c0 += u, c2 += e; else c1 += u, c3 += e;
    }
    c0 = __reduce_add_sync(~0u, c0);
    c1 = __reduce_add_sync(~0u, c1);
    c2 = __reduce_add_sync(~0u, c2);
    c3 = __reduce_add_sync(~0u, c3);
    if (lane == 0) cnt[warp] = make_int4(c0, c1, c2, c3);
  }
  cluster_barrier<R>();
  Ranks k = rank_warps<R>(s, cnt, need, rank);
  const unsigned below = (1u << lane) - 1u;
#pragma unroll
  for (int j = 0; j < KPT; ++j) {
    const int t0 = s.w0 + 32 * j, t = t0 + lane;
    if (t0 < s.w1) {
      const bool in = t < s.w1;
      bool keep = in && (int64_t)key[j] > over;
      const unsigned eq = __ballot_sync(~0u, in && need && key[j] == lim);
      if (eq >> lane & 1) keep = k.eq + __popc(eq & below) < need;
      k.eq += __popc(eq);
      if (keep && t < s.m) s.src[t] = t;
      const unsigned mv = __ballot_sync(~0u, keep && t >= s.m), ho = __ballot_sync(~0u, in && !keep && t < s.m);
      list_word(s, k, t0, mv, ho);
    }
  }
  fill_holes<R>(s, k.all_movers, rank);
}

// ---------------------------------------------------------------------------
// select, long slices: the keys do not fit, and most are far below the m-th
// largest.  A sample of 1024 keys a CTA gives a bound that, with five standard
// deviations to spare, fewer than m keys do not reach; one pass over the cache
// counts the keys from the bound on and lists them, per warp in slot order, in
// the workspace; all that follows reads the lists alone.  Where the bound was
// too high after all (the histogram tells), the pass is done again without one.
// grid: streams * R, cluster R; block 1024
// ---------------------------------------------------------------------------
template <int R>
__global__ void __launch_bounds__(ET, 1) evict_select_long_kernel(const __grid_constant__ EvictParams p) {
  // histograms: of the sample, and of each of two attempts at the pass
  __shared__ int hist[E_BINS + 2 * E_HIST];
  extern __shared__ int total[];          // R > 1: as hist, over all ranks
  __shared__ int ws[EW];
  __shared__ int4 cnt[EW];
  __shared__ int freed[EW];
  __shared__ int pick[3];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned below = (1u << lane) - 1u;
  const int rank = R > 1 ? (int)cl.block_rank() : 0;
  griddep_wait();
  griddep_launch();
  Slice s;
  if (!slice_of<R>(p, rank, s)) return;
  uint2* list = p.listed + (blockIdx.x / R) * p.list_slots + s.w0;
  for (int i = tid; i < E_BINS + 2 * E_HIST; i += ET) {
    hist[i] = 0;
    if constexpr (R > 1) total[i] = 0;
  }
  if constexpr (R > 1) cl.barrier_arrive();   // totals are zero
  __syncthreads();
  // sample: every (s1 - s0) / 1024-th slot
  const int64_t len = s.s1 - s.s0;
  if (len > 0) {
    const int t = s.s0 + (int)(len * tid / ET);
    atomicAdd(&hist[form_key(s, s.acc[t], s.pos[t]) >> 20], 1);
  }
  // slots below m that are not kept in the end stay marked
  for (int64_t t = rank * ET + tid; t < s.m; t += R * ET) s.src[t] = -1;
  if constexpr (R > 1) cl.barrier_wait();
  // every CTA with slots has ET samples; expected above the m-th key: part * m / n
  const int ctas = (s.n + s.sl - 1) / s.sl;
  const float want = (float)ctas * ET * ((float)s.m / (float)s.n);
  const int goal = (int)(want + 5.f * sqrtf(want) + 16.f);
  uint32_t floor_key = 0;
  if (goal < ctas * ET / 2) {
    pick_bin<R>(hist, total, E_BINS, goal, ws, pick);
    floor_key = (uint32_t)pick[0] << 20;
  } else {
    cluster_barrier<R>();                 // the marks come before any kept slot
  }
  int held = 0;                           // keys in this warp's list
  uint32_t lim = 0;
  int need = s.m;
  int* h0 = hist;
  int* t0h = total;
  const bool wide = ((reinterpret_cast<uintptr_t>(s.acc) | reinterpret_cast<uintptr_t>(s.pos)) & 15u) == 0;
#pragma unroll 1
  for (int attempt = 0; attempt < 2; ++attempt) {
    held = 0;
    h0 = hist + E_BINS + attempt * E_HIST;
    t0h = total + E_BINS + attempt * E_HIST;
    // 128 slots: lane i has 4 i .. 4 i + 3
    auto put4 = [&](const uint32_t (&k)[4], int t) {
      unsigned mine = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) mine |= (unsigned)(t + x < s.w1 && k[x] >= floor_key) << x;
      if (!__any_sync(~0u, mine)) return;
      int before = 0, all = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned w = __ballot_sync(~0u, mine >> x & 1);
        before += __popc(w & below);
        all += __popc(w);
      }
      before += held;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (mine >> x & 1) {
          atomicAdd(&h0[k[x] >> 20], 1);
          list[before++] = make_uint2(k[x], (uint32_t)(t + x));
        }
      held += all;
    };
    constexpr int U = 4;                  // groups in flight
    for (int g = s.w0; g < s.w1; g += 128 * U) {
      float4 a[U];
      int4 q[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int t = g + 128 * j + 4 * lane;
        a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        q[j] = make_int4(0, 0, 0, 0);
        if (wide && t + 4 <= s.w1) {
          a[j] = *reinterpret_cast<const float4*>(s.acc + t);
          q[j] = *reinterpret_cast<const int4*>(s.pos + t);
        } else {
          if (t < s.w1) a[j].x = s.acc[t], q[j].x = s.pos[t];
          if (t + 1 < s.w1) a[j].y = s.acc[t + 1], q[j].y = s.pos[t + 1];
          if (t + 2 < s.w1) a[j].z = s.acc[t + 2], q[j].z = s.pos[t + 2];
          if (t + 3 < s.w1) a[j].w = s.acc[t + 3], q[j].w = s.pos[t + 3];
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t k[4] = {form_key(s, a[j].x, q[j].x), form_key(s, a[j].y, q[j].y),
                               form_key(s, a[j].z, q[j].z), form_key(s, a[j].w, q[j].w)};
        put4(k, g + 128 * j + 4 * lane);
      }
    }
    __syncwarp();
    const int all = pick_bin<R>(h0, t0h, E_BINS, need, ws, pick);
    if (all >= need || floor_key == 0) break;
    floor_key = 0;                        // uniform in the cluster: all ranks see the same counts
  }
#pragma unroll
  for (int level = 0; level < 3; ++level) {
    constexpr int kShift[3] = {20, 10, 0}, kBase[3] = {0, E_BINS, E_BINS + E_BINS / 2};
    const int shift = kShift[level];
    if (level > 0) {
      int* hl = h0 + kBase[level];
#pragma unroll 4
      for (int i = lane; i < held; i += 32) {
        const uint32_t k = list[i].x;
        if ((k ^ lim) >> (shift + 10) == 0u) atomicAdd(&hl[(k >> shift) & 1023], 1);
      }
      pick_bin<R>(hl, t0h + kBase[level], E_BINS / 2, need, ws, pick);
    }
    lim |= (uint32_t)pick[0] << shift;
    need -= pick[1];
    if (pick[2] == need) {
      need = 0;
      break;
    }
  }
  const int64_t over = need == 0 ? (int64_t)lim - 1 : (int64_t)lim;
  {
    int c0 = 0, c1 = 0, c2 = 0, c3 = 0;
#pragma unroll 4
    for (int i = lane; i < held; i += 32) {
      const uint2 v = list[i];
      const int u = (int64_t)v.x > over, e = need && v.x == lim;
      if ((int)v.y < s.m) c0 += u, c2 += e; else c1 += u, c3 += e;
    }
    c0 = __reduce_add_sync(~0u, c0);
    c1 = __reduce_add_sync(~0u, c1);
    c2 = __reduce_add_sync(~0u, c2);
    c3 = __reduce_add_sync(~0u, c3);
    if (lane == 0) cnt[warp] = make_int4(c0, c1, c2, c3);
  }
  cluster_barrier<R>();
  Ranks k = rank_warps<R>(s, cnt, need, rank);
#pragma unroll 2
  for (int i0 = 0; i0 < held; i0 += 32) {
    const bool in = i0 + lane < held;
    const uint2 v = in ? list[i0 + lane] : make_uint2(0u, 0u);
    const int t = (int)v.y;
    bool keep = in && (int64_t)v.x > over;
    const unsigned eq = __ballot_sync(~0u, in && need && v.x == lim);
    if (eq >> lane & 1) keep = k.eq + __popc(eq & below) < need;
    k.eq += __popc(eq);
    if (keep && t < s.m) s.src[t] = t;
    const unsigned mv = __ballot_sync(~0u, keep && t >= s.m);
    const int im = k.movers + __popc(mv & below);
    if ((mv >> lane & 1) && im >= 0 && im < s.m) s.movers[im] = t;
    k.movers += __popc(mv);
  }
  cluster_barrier<R>();                   // kept slots are unmarked, movers listed
  // freed slots, ranked over an even share of slots 0 .. m - 1 for every warp
  const int share = ((s.m + R * EW - 1) / (R * EW) + 31) / 32 * 32;
  const int f0 = min(s.m, (rank * EW + warp) * share), f1 = min(s.m, f0 + share);
  int mine = 0;
#pragma unroll 4
  for (int t = f0 + lane; t < f1; t += 32) mine += __ldcg(s.src + t) < 0;
  mine = __reduce_add_sync(~0u, mine);
  if (lane == 0) freed[warp] = mine;
  cluster_barrier<R>();
  int rank_of = 0;                        // freed slots before this warp's
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int v = q <= rank ? (R > 1 ? *cl.map_shared_rank(&freed[lane], q) : freed[lane]) : 0;
    rank_of += __reduce_add_sync(~0u, q < rank || (q == rank && lane < warp) ? v : 0);
  }
  for (int t = f0 + lane; t - lane < f1; t += 32) {
    const bool ho = t < f1 && __ldcg(s.src + t) < 0;
    const unsigned w = __ballot_sync(~0u, ho);
    const int i = rank_of + __popc(w & below);
    if (ho && i < min(k.all_movers, s.m)) s.src[t] = __ldcg(s.movers + i);
    rank_of += __popc(w);
  }
  if constexpr (R > 1) cl.sync();         // no rank's counts are read any more
}

// ---------------------------------------------------------------------------
// move: rows of moved tokens, accumulated weights and positions of all kept
// ones, new lengths.  A group of row_bytes / 16 lanes copies a row.
// grid: streams * chunks of MS slots
// ---------------------------------------------------------------------------
constexpr int MT = 256, MS = 128;

__global__ void __launch_bounds__(MT) evict_move_kernel(const __grid_constant__ EvictParams p, int chunks) {
  __shared__ int64_t to_row[MS], from_row[MS];   // -1: stays
  const int64_t stream = blockIdx.x / chunks;
  const int c0 = (int)(blockIdx.x - stream * chunks) * MS;
  const int b = (int)(stream / p.H), h = (int)(stream - (int64_t)b * p.H);
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch();
  int moved = 0;
  if (tid < MS) {
    const int t = c0 + tid;
    int s = t < p.budget ? p.src[stream * p.budget + t] : -1;
    if (s >= p.limit) s = -1;
    int64_t to = -1, from = -1;
    if (s >= 0 && s != t) {
      const int32_t* tab = p.table + b * p.table_stride;
      const int pt = tab[t / p.ps], pf = tab[s / p.ps];
      if (pt >= 0 && pt < p.n_pages && pf >= 0 && pf < p.n_pages) {
        to = ((int64_t)pt * p.H + h) * p.ps + t % p.ps;
        from = ((int64_t)pf * p.H + h) * p.ps + s % p.ps;
        moved = 1;
      } else if (p.status) {
        atomicOr(p.status, DEV_ERR_CHECK);
      }
    }
    to_row[tid] = to;
    from_row[tid] = from;
    if (s >= 0) {
      const int64_t i = stream * p.meta_stride + s, o = stream * p.out_stride + t;
      if (s != t || p.acc_out != p.acc) p.acc_out[o] = p.acc[i];
      if (s != t || p.pos_out != p.pos) p.pos_out[o] = p.pos[i];
    }
    if (h == 0 && t == 0) {
      const int n = evict_len(p, b);
      p.lens_out[b] = min(n, p.budget);
    }
  }
  if (!__syncthreads_or(moved)) return;
  const int L = p.row_bytes / 16;         // lanes of a row: 4, 8, 16 or 32
  const int e = tid % L;
  // 2 MS rows (keys, then values), MT / L at a time, 4 in flight a thread
  for (int i0 = tid / L; i0 < 2 * MS; i0 += 4 * (MT / L)) {
    uint4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + x * (MT / L);
      if (i < 2 * MS && to_row[i % MS] >= 0)
        v[x] = *reinterpret_cast<const uint4*>((i < MS ? p.kp : p.vp) + from_row[i % MS] * p.row_bytes + 16 * e);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = i0 + x * (MT / L);
      if (i < 2 * MS && to_row[i % MS] >= 0)
        *reinterpret_cast<uint4*>((i < MS ? p.kp : p.vp) + to_row[i % MS] * p.row_bytes + 16 * e) = v[x];
    }
  }
}

}  // namespace

namespace {

// Slots of a CTA of a stream of n tokens.
int64_t evict_slice(int64_t n, int R) { return ((n + R - 1) / R + ET - 1) / ET * ET; }

template <int R>
cudaError_t select_r(const EvictParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)p.B * p.H * R));
  const int64_t sl = evict_slice(p.limit, R);
  if (sl <= 8 * ET) return launch_kernel(evict_select_kernel<R, 8>, grid, dim3(ET), 0, st, true, R, p);
  if (sl <= E_SHORT) return launch_kernel(evict_select_kernel<R, E_SHORT / ET>, grid, dim3(ET), 0, st, true, R, p);
  const int totals = R > 1 ? (E_BINS + 2 * E_HIST) * (int)sizeof(int) : 0;
  const cudaError_t e = cudaFuncSetAttribute(evict_select_long_kernel<R>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, totals);
  if (e != cudaSuccess) return e;
  return launch_kernel(evict_select_long_kernel<R>, grid, dim3(ET), totals, st, true, R, p);
}

}  // namespace

int64_t evict_list_slots(int64_t limit, int R) {
  return evict_slice(limit, R) <= E_SHORT ? 0 : limit;
}

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t st) {
  switch (p.R) {
    case 1: return select_r<1>(p, st);
    case 2: return select_r<2>(p, st);
    case 4: return select_r<4>(p, st);
    default: return select_r<8>(p, st);
  }
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t st) {
  const int chunks = ((p.budget < p.limit ? p.budget : p.limit) + MS - 1) / MS;
  return launch_kernel(evict_move_kernel, dim3((unsigned)((int64_t)p.B * p.H * chunks)), dim3(MT), 0, st,
                       true, 0, p, chunks);
}

}  // namespace mkv
