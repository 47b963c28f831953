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
constexpr int E_MAX_R = 8;
constexpr int E_CAP = 40960;              // keys of a slice held in shared memory
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

// ---------------------------------------------------------------------------
// grid: streams * R, cluster R; block 1024; dynamic smem: the slice's keys
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(ET) evict_select_kernel(const __grid_constant__ EvictParams p,
                                                          int key_cap) {
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ uint32_t keys[];
  __shared__ int hist[E_BINS];
  __shared__ int ws[EW];
  __shared__ int cnt[EW][4];              // per warp: above / equal keys, below and from slot m
  __shared__ int pick[3];                 // bin, keys above it, keys in it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.R, rank = R > 1 ? (int)cl.block_rank() : 0;
  const int64_t stream = blockIdx.x / R;
  const int b = (int)(stream / p.H), h = (int)(stream - (int64_t)b * p.H);
  const int n = evict_len(p, b), m = p.budget;
  int32_t* src = p.src + stream * m;
  griddep_launch();
  if (h == 0 && rank == 0 && tid == 0 && p.status && p.lens[b] != n) atomicOr(p.status, DEV_ERR_CHECK);
  if (n <= m) {                           // nothing to evict (uniform in the cluster)
    for (int64_t i = rank * ET + tid; i < m; i += (int64_t)R * ET) src[i] = i < n ? (int)i : -1;
    return;
  }
  const float* acc = p.acc + stream * p.meta_stride;
  const int32_t* pos = p.pos + stream * p.meta_stride;
  const int64_t from = (int64_t)p.next_pos[b] - p.recent;
  auto compute = [&](int t) -> uint32_t {
    const int q = pos[t];
    const float a = acc[t];
    if (q < p.sink || q >= from) return KEY_SAFE;
    return a > 0.f ? __float_as_uint(a) : 0u;
  };
  // this CTA's slots; a warp's share is a multiple of 32 slots
  const int sl = ((n + R - 1) / R + ET - 1) / ET * ET;
  const int s0 = min(n, rank * sl), s1 = min(n, s0 + sl);
  const int held = min(s1 - s0, key_cap);
#pragma unroll 4
  for (int i = tid; i < held; i += ET) keys[i] = compute(s0 + i);
  auto key = [&](int t) -> uint32_t { return t - s0 < held ? keys[t - s0] : compute(t); };
  auto sync_all = [&]() {
    if (R > 1) cl.sync(); else __syncthreads();
  };

  // the m-th largest key, 11 + 10 + 10 bits at a time.  `above`: keep keys > lim;
  // `need`: of those equal to lim, the lowest slots
  uint32_t prefix = 0, lim = 0;
  int need = m;
  int shift = 20;
  for (int level = 0; level < 3; ++level) {
    const int bins = level == 0 ? 2048 : 1024;
    const uint32_t hi_mask = level == 0 ? 0u : 0xffffffffu << (shift + 10);
    for (int i = tid; i < bins; i += ET) hist[i] = 0;
    __syncthreads();
    for (int t = s0 + tid; t < s1; t += ET) {
      const uint32_t k = key(t);
      if ((k & hi_mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
    }
    sync_all();
    // counts of bins from the top: thread i takes bins (bins - 1 - i PER ...)
    int mine[2] = {0, 0};
    const int per = bins / ET;
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (x < per) {
        const int bin = bins - 1 - (tid * per + x);
        if (R > 1)
          for (int q = 0; q < R; ++q) mine[x] += *cl.map_shared_rank(&hist[bin], q);
        else
          mine[x] = hist[bin];
      }
    int all;
    int before = block_prefix(mine[0] + mine[1], ws, &all);
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (x < per) {
        if (before < need && before + mine[x] >= need) {
          pick[0] = bins - 1 - (tid * per + x);
          pick[1] = before;
          pick[2] = mine[x];
        }
        before += mine[x];
      }
    sync_all();                           // pick is set; every rank has read the histograms
    prefix |= (uint32_t)pick[0] << shift;
    need -= pick[1];
    const bool all_in = pick[2] == need;
    __syncthreads();                      // pick may be written again
    if (all_in || level == 2) {
      lim = prefix;
      if (all_in) {                       // the whole bin is kept: no key equals lim's predecessor
        need = 0;
        break;
      }
    }
    shift -= 10;
  }
  const bool whole_bin = need == 0;       // keep keys >= lim, else > lim and `need` equal ones
  auto above = [&](uint32_t k) { return whole_bin ? k >= lim : k > lim; };
  auto equal = [&](uint32_t k) { return !whole_bin && k == lim; };

  // counts of this warp's run of slots
  const int wl = sl / EW;
  const int w0 = min(s1, s0 + warp * wl), w1 = min(s1, w0 + wl);
  int ab[2] = {0, 0}, eq[2] = {0, 0};
#pragma unroll 2
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t k = t < w1 ? key(t) : 0u;
    const bool up = t < w1 && above(k), same = t < w1 && equal(k);
    const unsigned lo = __ballot_sync(~0u, t < m);
    const unsigned u = __ballot_sync(~0u, up), s = __ballot_sync(~0u, same);
    ab[0] += __popc(u & lo), ab[1] += __popc(u & ~lo);
    eq[0] += __popc(s & lo), eq[1] += __popc(s & ~lo);
  }
  if (lane == 0) cnt[warp][0] = ab[0], cnt[warp][1] = ab[1], cnt[warp][2] = eq[0], cnt[warp][3] = eq[1];
  sync_all();
  // equal keys, movers and freed slots of all warps before this one, in slot order
  int eq_before = 0, movers = 0, holes = 0, all_movers = 0;
  {
    const int total = R * EW, me = rank * EW + warp;
    int run_eq = 0, run_mv = 0, run_ho = 0;
    for (int g = 0; g < total; g += 32) {
      const int w = g + lane;             // all entries of one rank: EW = 32
      const int* e = R > 1 ? cl.map_shared_rank(&cnt[lane][0], g / EW) : &cnt[lane][0];
      const int a1 = e[1], e0 = e[2], e1 = e[3], a0 = e[0];
      int inc = e0 + e1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += u;
      }
      const int eb = run_eq + inc - (e0 + e1);
      const int k0 = min(max(need - eb, 0), e0), k1 = min(max(need - eb - e0, 0), e1);
      const int first = min(n, (w / EW) * sl) + (w % EW) * wl;
      const int last = min(first + wl, min(n, (w / EW) * sl + sl));
      const int slots_lo = max(0, min(last, m) - first);
      const int mv = a1 + k1, ho = slots_lo - a0 - k0;
      int im = mv, ih = ho;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, im, o), v = __shfl_up_sync(~0u, ih, o);
        if (lane >= o) im += u, ih += v;
      }
      if (g == (me & ~31)) {
        eq_before = __shfl_sync(~0u, eb, me & 31);
        movers = run_mv + __shfl_sync(~0u, im - mv, me & 31);
        holes = run_ho + __shfl_sync(~0u, ih - ho, me & 31);
      }
      run_eq += __shfl_sync(~0u, inc, 31);
      run_mv += __shfl_sync(~0u, im, 31);
      run_ho += __shfl_sync(~0u, ih, 31);
    }
    all_movers = run_mv;
  }
  int32_t* mover_list = p.lists + stream * 2 * m;
  int32_t* hole_list = mover_list + m;
  const unsigned below = (1u << lane) - 1u;
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const bool in = t < w1;
    const uint32_t k = in ? key(t) : 0u;
    const unsigned same = __ballot_sync(~0u, in && equal(k));
    const bool keep = in && (above(k) || ((same >> lane & 1) && eq_before + __popc(same & below) < need));
    const unsigned mv = __ballot_sync(~0u, keep && t >= m), ho = __ballot_sync(~0u, in && !keep && t < m);
    // The ranks are below m; the checks hold that too where another stream
    // writes the weights meanwhile and the passes see different keys.
    const int im = movers + __popc(mv & below), ih = holes + __popc(ho & below);
    if (keep && t >= m && im < m) mover_list[im] = t;
    if (in && t < m) {
      if (keep)
        src[t] = t;
      else if (ih >= 0 && ih < m)
        hole_list[ih] = t;
    }
    eq_before += __popc(same);
    movers += __popc(mv);
    holes += __popc(ho);
  }
  sync_all();                             // lists are complete (and no rank's counts are read any more)
  for (int i = rank * ET + tid; i < min(all_movers, m); i += R * ET) {
    const int t = hole_list[i];
    if (t >= 0 && t < m) src[t] = mover_list[i];
  }
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

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t st) {
  const int sl = ((p.limit + p.R - 1) / p.R + ET - 1) / ET * ET;
  const int cap = sl < E_CAP ? sl : E_CAP;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       E_CAP * 4);
  if (e != cudaSuccess) return e;
  return launch_kernel(evict_select_kernel, dim3((unsigned)((int64_t)p.B * p.H * p.R)), dim3(ET),
                       (size_t)cap * 4, st, false, p.R, p, cap);
}

cudaError_t launch_evict_move(const EvictParams& p, cudaStream_t st) {
  const int chunks = ((p.budget < p.limit ? p.budget : p.limit) + MS - 1) / MS;
  return launch_kernel(evict_move_kernel, dim3((unsigned)((int64_t)p.B * p.H * chunks)), dim3(MT), 0, st,
                       true, 0, p, chunks);
}

}  // namespace mkv
