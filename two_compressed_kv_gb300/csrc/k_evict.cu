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
// traffic per moved token.
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
  s.movers = p.lists + stream * 2 * s.m;
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

// The bin of the `need`-th largest key, from the ranks' histograms of `bins`
// bins: pick = {bin, keys in bins above, keys in it}.  Returns the keys in all.
// Ends with a block barrier.
template <int R>
__device__ __forceinline__ int pick_bin(int* hist, int bins, int need, int* ws, int* pick) {
  cg::cluster_group cl = cg::this_cluster();
  constexpr int MAXPER = E_BINS / ET;
  const int per = bins / ET;
  int mine[MAXPER] = {}, sum = 0;
#pragma unroll
  for (int x = 0; x < MAXPER; ++x)
    if (x < per) {
      const int bin = bins - 1 - ((int)threadIdx.x * per + x);   // from the top
      int v[R];
#pragma unroll
      for (int q = 0; q < R; ++q) v[q] = R > 1 ? *cl.map_shared_rank(&hist[bin], q) : hist[bin];
#pragma unroll
      for (int q = 0; q < R; ++q) mine[x] += v[q];
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
// histogram of its own and costs one cluster barrier: nothing that another rank
// still reads is written again.
// grid: streams * R, cluster R; block 1024
// ---------------------------------------------------------------------------
template <int R, int KPT>
__global__ void __launch_bounds__(ET, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int hist[E_BINS + 2 * (E_BINS / 2)];
  __shared__ int ws[EW];
  __shared__ int4 cnt[EW];
  __shared__ int pick[3];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = R > 1 ? (int)cg::this_cluster().block_rank() : 0;
  griddep_launch();
  Slice s;
  if (!slice_of<R>(p, rank, s)) return;
  uint32_t key[KPT];
  {
    float a[KPT];
    int q[KPT];
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int t = s.w0 + 32 * j + lane;
      if (t < s.w1) a[j] = s.acc[t], q[j] = s.pos[t];
    }
    for (int i = tid; i < 2 * E_BINS; i += ET) hist[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      key[j] = 0;
      if (s.w0 + 32 * j + lane < s.w1) {
        key[j] = form_key(s, a[j], q[j]);
        atomicAdd(&hist[key[j] >> 20], 1);
      }
    }
  }
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
    cluster_barrier<R>();
    pick_bin<R>(hl, level == 0 ? E_BINS : E_BINS / 2, need, ws, pick);
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
    if (lane == 0) cnt[tid >> 5] = make_int4(c0, c1, c2, c3);
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
  __shared__ int sample[E_BINS];
  __shared__ int hist[2][E_BINS + 2 * (E_BINS / 2)];
  __shared__ int ws[EW];
  __shared__ int4 cnt[EW];
  __shared__ int pick[3];
  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned below = (1u << lane) - 1u;
  const int rank = R > 1 ? (int)cg::this_cluster().block_rank() : 0;
  griddep_launch();
  Slice s;
  if (!slice_of<R>(p, rank, s)) return;
  uint2* list = p.listed + (blockIdx.x / R) * p.list_slots + s.w0;
  for (int i = tid; i < E_BINS; i += ET) sample[i] = 0;
  for (int i = tid; i < 4 * E_BINS; i += ET) (&hist[0][0])[i] = 0;
  __syncthreads();
  // sample: slot i of every (s1 - s0) / 1024
  const int64_t len = s.s1 - s.s0;
  const int mine_at = s.s0 + (int)(len * tid / ET);
  const bool sampled = len > 0;
  if (sampled) atomicAdd(&sample[form_key(s, s.acc[mine_at], s.pos[mine_at]) >> 20], 1);
  for (int t = s.w0 + lane; t < min(s.w1, s.m); t += 32) s.src[t] = -1;    // marks freed slots
  cluster_barrier<R>();
  // every CTA with slots has ET samples; expected above the m-th key: part * m / n
  const int ctas = (s.n + s.sl - 1) / s.sl;
  const float want = (float)ctas * ET * ((float)s.m / (float)s.n);
  const int goal = (int)(want + 5.f * sqrtf(want) + 16.f);
  uint32_t floor_key = 0;
  if (goal < ctas * ET / 2) {
    pick_bin<R>(sample, E_BINS, goal, ws, pick);
    floor_key = (uint32_t)pick[0] << 20;
  }
  int held = 0;                           // keys in this warp's list
  uint32_t lim = 0;
  int need = s.m;
  int* h0 = hist[0];
#pragma unroll 1
  for (int attempt = 0; attempt < 2; ++attempt) {
    held = 0;
    h0 = hist[attempt];
    auto put = [&](uint32_t k, int t, bool in) {
      if (in) atomicAdd(&h0[k >> 20], 1);
      const unsigned w = __ballot_sync(~0u, in);
      if (in) list[held + __popc(w & below)] = make_uint2(k, (uint32_t)t);
      held += __popc(w);
    };
    constexpr int U = 8;                  // words of 32 slots in flight
    for (int t0 = s.w0; t0 < s.w1; t0 += 32 * U) {
      float a[U];
      int q[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int t = t0 + 32 * j + lane;
        a[j] = 0.f, q[j] = 0;
        if (t < s.w1) a[j] = s.acc[t], q[j] = s.pos[t];
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int t = t0 + 32 * j + lane;
        const uint32_t k = form_key(s, a[j], q[j]);
        const bool in = t < s.w1 && k >= floor_key;
        if (__any_sync(~0u, in)) put(k, t, in);
      }
    }
    __syncwarp();
    cluster_barrier<R>();
    const int all = pick_bin<R>(h0, E_BINS, need, ws, pick);
    if (all >= need || floor_key == 0) break;
    floor_key = 0;                        // uniform in the cluster: all ranks see the same counts
  }
#pragma unroll
  for (int level = 0; level < 3; ++level) {
    constexpr int kShift[3] = {20, 10, 0}, kBase[3] = {0, E_BINS, E_BINS + E_BINS / 2};
    const int shift = kShift[level];
    int* hl = h0 + kBase[level];
    if (level > 0) {
#pragma unroll 4
      for (int i = lane; i < held; i += 32) {
        const uint32_t k = list[i].x;
        if ((k ^ lim) >> (shift + 10) == 0u) atomicAdd(&hl[(k >> shift) & 1023], 1);
      }
      cluster_barrier<R>();
      pick_bin<R>(hl, E_BINS / 2, need, ws, pick);
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
    if (lane == 0) cnt[tid >> 5] = make_int4(c0, c1, c2, c3);
  }
  cluster_barrier<R>();
  Ranks k = rank_warps<R>(s, cnt, need, rank);
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
  __syncwarp();
  // slots below m that were not kept; the warp's own marks
#pragma unroll 4
  for (int t0 = s.w0; t0 < min(s.w1, s.m); t0 += 32) {
    const int t = t0 + lane;
    const unsigned ho = __ballot_sync(~0u, t < min(s.w1, s.m) && s.src[t] < 0);
    list_word(s, k, t0, 0u, ho);
  }
  fill_holes<R>(s, k.all_movers, rank);
}

// ---------------------------------------------------------------------------
// move: rows of moved tokens, accumulated weights and positions of all kept
// ones, new lengths.  A group of row_bytes / 16 lanes copies a row.
// grid: streams * chunks of MS slots
// ---------------------------------------------------------------------------
constexpr int MT = 256, MS = 64;

__global__ void __launch_bounds__(MT) evict_move_kernel(const __grid_constant__ EvictParams p, int chunks) {
  __shared__ int32_t sm_src[MS];
  __shared__ int64_t to_row[MS], from_row[MS];   // -1: stays
  const int64_t stream = blockIdx.x / chunks;
  const int c0 = (int)(blockIdx.x - stream * chunks) * MS;
  const int b = (int)(stream / p.H), h = (int)(stream - (int64_t)b * p.H);
  const int tid = threadIdx.x;
  griddep_wait();
  int moved = 0;
  if (tid < MS) {
    const int t = c0 + tid;
    int s = t < p.budget ? p.src[stream * p.budget + t] : -1;
    if (s >= p.limit) s = -1;
    sm_src[tid] = s;
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
  if (sl <= 8 * ET) return launch_kernel(evict_select_kernel<R, 8>, grid, dim3(ET), 0, st, false, R, p);
  if (sl <= E_SHORT) return launch_kernel(evict_select_kernel<R, E_SHORT / ET>, grid, dim3(ET), 0, st, false, R, p);
  return launch_kernel(evict_select_long_kernel<R>, grid, dim3(ET), 0, st, false, R, p);
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
