// Attention of one new token per sequence over a paged cache: the streaming
// kernel, included by one translation unit per head dimension.
//
// For a stream (sequence b, KV head h) with g query heads and n cached tokens:
//   z_it = scale q_i . k_t,  p_it = exp(z_it - max_t z_it),
//   o_i = sum_t p_it v_t / sum_t p_it,
// in one pass over the tokens with a running maximum m and sum l: when m grows
// by d, l and o are multiplied by exp(-d).  Parts of a stream are joined the
// same way.
//
// What bounds it: each key and value row is used once for at most 16 query
// heads, 2 g operations per byte (fp16), so DRAM bounds it and the kernel is
// built to keep enough copies in flight with few instructions per byte:
//   - a warp works alone on blocks of 16 tokens; no barrier between warps until
//     its part of a stream is done;
//   - the 16 rows of a block come by one TMA copy for keys and one for values
//     into the warp's own ring in shared memory, 128-byte swizzled;
//   - transposed products, S^T = K Q^T and O^T = V^T P^T as m16n8k16: tokens,
//     then channels, are the 16 rows, and 8 query heads fill the 8 columns, so
//     that no row is padding (with heads as rows, half of the work and of the
//     accumulators is).  16-bit rows reach the fragments by ldmatrix, values
//     transposed on the way; of e4m3 rows a lane reads 16 bytes, pairs tokens by
//     byte permutes and converts to fp16, exactly.  There row n of a fragment is
//     token n ^ 4 (n & 1) of 8, which keeps the reads free of bank conflicts.
//     tcgen05 would need the operands unpacked back into shared memory, and
//     m16n8k16 is far from its rate here;
//   - P in 16 bits would cost half the output's precision, so it goes in as a
//     high and a low part.  Probabilities carry a factor 2^12, which cancels, so
//     that small ones stay normal in fp16 and the reference of the exponents need
//     not follow every new maximum: up to 2^3 above it still fits.
//
// Measured: 32768 tokens, batch 4, 8 KV heads, fp16: 85 us in the kernel, 6.3 TB/s,
// 94 % of a copy's rate, 88 us with the join; 131072, batch 8, bf16, with weights:
// 695 us, 6.3 TB/s; a ragged batch of 256 e4m3 streams: 75.7 us, 4.8 TB/s.  There no
// unit is full (issue 0.46 a cycle, tensor pipe 24 %, DRAM 67 % of its peak): the
// chains of 64 conversions and 24 products per 4 KB, at three warps a scheduler, and
// the starts of parts take the time.
#pragma once

#include <cooperative_groups.h>
#include <math_constants.h>

#include "decode_common.cuh"
#include "paged_internal.cuh"
#include "ptx.cuh"
#include "tc05.cuh"

namespace mkv {
namespace {

// m16n8k16 products with fp32 accumulation.  Not volatile: the compiler may
// interleave them with the loads and conversions of the next step.
template <bool BF16>
__device__ __forceinline__ void mma_acc(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 values as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Two probabilities as 16-bit pairs: rounded, what the rounding left, rounded,
// and (bf16) what that left.
template <bool BF16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo, uint32_t& rest) {
  if constexpr (BF16) {
    auto part = [&](float& x, float& y) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      x -= __low2float(h);
      y -= __high2float(h);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    hi = part(a, b);
    lo = part(a, b);
    rest = part(a, b);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

// Four 8 x 8 tiles of 16-bit elements, rows at the lanes' addresses (lanes 8 i ..
// 8 i + 7: tile i); lane 4 r + c gets elements 2 c, 2 c + 1 of row r, or (TRANS)
// of column r.  Ordered with the waits on the ring, otherwise free to move.
template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// An 8 x 8 tile of 16-bit elements, a row's pair a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}

template <int CT, int D, bool WIDE, int NW>
struct PA {
  static constexpr int ES = CT == MKV_DT_E4M3 ? 1 : 2;
  static constexpr bool BF16 = CT == MKV_DT_BF16;
  static constexpr int ROW = D * ES;                       // bytes of a row
  static constexpr int SW = ROW < 128 ? ROW : 128;         // swizzled width
  static constexpr int KL = ROW / 64;                      // e4m3: 16-byte pieces of a key row per lane
  static constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16;   // e4m3: bytes of a value piece
  static constexpr int VL = ROW / (8 * VB);                // e4m3: value pieces of a row per lane
  static constexpr int NH = WIDE ? 2 : 1;                  // groups of 8 heads
  static constexpr int KS = D / 16;                        // contraction steps of S^T, row tiles of O^T
  static constexpr int STAGE = 2 * PA_BLOCK * ROW;         // bytes of one block's keys and values
  static constexpr int U = STAGE >= 8192 ? 1 : 2;          // blocks of a step
  static constexpr int STAGES = STAGE >= 8192 ? 3 : STAGE >= 4096 ? 4 : 8;
  static_assert(STAGES % U == 0, "a step's slots do not wrap");
  static constexpr int HR = 8 * NH;                        // head rows
  static constexpr int MERGE = NW * HR * (D + 4) * 4;
  static constexpr int OWN = HR * D * 4;                   // cluster: this CTA's sums, behind the merge area
  static constexpr int RING = NW * STAGES * STAGE;
  static constexpr int SMEM = (RING > MERGE + OWN ? RING : MERGE + OWN) + 1024;   // and its alignment
  static constexpr int CTAS = NW == 8 ? 1 : paged_ctas(ROW);   // per SM
  static_assert(CTAS * (SMEM + 9 * 1024) <= 228 * 1024, "resident CTAs' shared memory");
};

// Byte offset of 16-byte piece `piece` (of the first SW bytes) of row `row` in a
// block's keys or values: [row / SW columns][16 rows][SW bytes], pieces of a row
// permuted by the TMA swizzle (128 bytes: by row mod 8; 64 bytes: by row / 2 mod
// 4).  Neither changes from row to row + 8.
template <int SW>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return SW == 128 ? (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4))
                   : (uint32_t)(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}
// From the offset `at` of a piece: that of the piece `by` further, where `by` has
// no bit in common with the piece's number in its 128 bytes.
__device__ __forceinline__ uint32_t piece_on(uint32_t at, int by) {
  return (at ^ ((uint32_t)(by & 7) << 4)) + (uint32_t)(by >> 3) * (PA_BLOCK * 128);
}

// ---------------------------------------------------------------------------
// grid: split ? 3 G : streams * cluster; cluster (cluster, 1, 1); block: NW warps; dynamic smem PA::SMEM
// ---------------------------------------------------------------------------
template <int CT, int D, bool WIDE, int NW, bool THIRD>
__global__ void __launch_bounds__(NW * 32, PA<CT, D, WIDE, NW>::CTAS)
    paged_attn_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using C = PA<CT, D, WIDE, NW>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);   // the swizzle goes by address bits 7..9
  __shared__ uint64_t full[NW][C::STAGES];
  __shared__ int64_t pre[PA_MAX_B + 1];        // split: load before each sequence,
  __shared__ int len_of[PA_MAX_B];             // and its length
  __shared__ float sm_m[NW][C::HR], sm_l[NW][C::HR];
  __shared__ int64_t warp_sum[NW];
  __shared__ float2 own_ml[C::HR];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;       // fragment row and column pair
  constexpr int NH = C::NH;
  constexpr bool E4 = CT == MKV_DT_E4M3;
  uint8_t* const ring_p = smem + warp * (C::STAGES * C::STAGE);
  // where this lane reads.  ldmatrix: keys, tokens 0..7, 8..15 of the first and
  // second 8 channels; values, 8 channels of tokens 0..7, the next 8, then 8..15.
  // e4m3: key row of token r, value rows of its column pair's tokens.
  const uint32_t k_at = E4 ? piece_at<C::SW>(r ^ ((r & 1) << 2), c)
                           : piece_at<128>((lane & 7) + (lane & 8), lane >> 4);
  const uint32_t v_at = E4 ? piece_at<C::SW>(2 * c, C::VB == 16 ? r : r >> 1) + (C::VB == 16 ? 0 : 8 * (r & 1))
                           : piece_at<128>((lane & 7) + ((lane >> 1) & 8), (lane >> 3) & 1);
  const uint32_t v_at1 = E4 ? piece_at<C::SW>((2 * c + 1) ^ 4, C::VB == 16 ? r : r >> 1) + (C::VB == 16 ? 0 : 8 * (r & 1))
                            : 0u;
  // token of this lane's first row of S^T (the second is 8 further)
  const int tok_r = E4 ? r ^ ((r & 1) << 2) : r;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < C::STAGES; ++k) mbar_init(&full[warp][k], 1);
    mbar_init_fence();
  }
  __syncwarp();
  uint32_t phases = 0;                         // bit of a ring slot: parity of its next fill
  uint32_t pending = 0;                        // bit of a ring slot: a copy into it is in flight
  bool gave_up = false;                        // a bounded wait ran out: outputs undefined

  griddep_wait();                              // lengths and caches may come from the kernel before
  griddep_launch();                            // the join's prologue may start; it waits for the end
  // this CTA's share of the load, counted over all streams
  int64_t g0 = 0, g1 = 0, at = 0;
  int b = 0;
  if (p.split) {
    // prefix sums of the sequences' load: each thread a run of sequences
    const int run = (p.B + NW * 32 - 1) / (NW * 32);
    int64_t sum = 0;
    for (int k = 0; k < run; ++k) {
      const int i = tid * run + k;
      if (i < p.B) {
        len_of[i] = paged_len(p, i);
        sum += paged_load(p, len_of[i]) * p.H;
      }
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int64_t base = inc - sum;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int k = 0; k < run; ++k) {
      const int i = tid * run + k;
      if (i < p.B) {
        pre[i] = base;
        base += paged_load(p, len_of[i]) * p.H;
      }
      if (i == p.B - 1) pre[p.B] = base;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i <= p.B; i += NW * 32) p.pre[i] = pre[i];   // for the join
    const PagedShares shares(p, pre[p.B]);
    g0 = shares.first(blockIdx.x);
    g1 = shares.first(blockIdx.x + 1);
    if (g0 >= g1) return;
    int lo = 0, hi = p.B - 1;                  // last b with pre[b] <= g0 that has blocks
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= g0) lo = mid; else hi = mid - 1;
    }
    b = lo;
    at = g0;
  }

  while (true) {
    // next piece: blocks [j0, j1) of stream (b, h)
    int h, j0, j1, n, nb;
    if (p.split) {
      if (at >= g1) break;
      while (pre[b + 1] <= at) ++b;
      n = len_of[b];
      nb = (n + PA_BLOCK - 1) / PA_BLOCK;
      const int64_t off = at - pre[b];
      const int load = (int)paged_load(p, n);
      h = (int)div_small(off, load);
      const int v0 = (int)(off - (int64_t)h * load), v1 = (int)min((int64_t)load, v0 + (g1 - at));
      at += v1 - v0;
      j0 = max(0, v0 - p.piece_load);
      j1 = v1 - p.piece_load;
      if (j1 <= j0) continue;
    } else {
      const int s = blockIdx.x / p.cluster, rank = blockIdx.x - s * p.cluster;
      b = s / p.H;
      h = s - b * p.H;
      n = paged_len(p, b);
      nb = (n + PA_BLOCK - 1) / PA_BLOCK;
      j0 = (int)((int64_t)nb * rank / p.cluster);
      j1 = (int)((int64_t)nb * (rank + 1) / p.cluster);
      if (rank == 0 && h == 0 && tid == 0 && p.status && p.lens[b] != n) atomicOr(p.status, DEV_ERR_CHECK);
    }
    if (p.split && h == 0 && j0 == 0 && tid == 0 && p.status && p.lens[b] != n)
      atomicOr(p.status, DEV_ERR_CHECK);
    const int64_t stream = (int64_t)b * p.H + h;

    // this warp's blocks: j0 + warp, + 4, ...; lane i holds the pool row of
    // the i-th of the next 32 (in blocks of 16 rows; -1: page outside the cache)
    const int count = gave_up ? 0 : max(0, (j1 - j0 - warp + NW - 1) / NW);
    auto entries = [&](int first) {
      const int j = j0 + warp + NW * (first + lane);
      int e = -1;
      if (first + lane < count) {
        const int pg = j / p.bpp;
        const int page = p.table[(int64_t)b * p.table_stride + pg];
        if (page >= 0 && page < p.n_pages)
          e = (page * p.H + h) * p.bpp + (j - pg * p.bpp);
        else if (p.status)
          atomicOr(p.status, DEV_ERR_CHECK);
      }
      return e;
    };
    int ent = entries(0), ent_next = entries(32);
    int valid_bits = 0;                        // bit of a ring slot: its page is there
    auto issue = [&](int i, int slot) {
      if (i >= count) return;
      if ((i & 31) == 0 && i > 0) {
        ent = ent_next;
        ent_next = entries(i + 32);
      }
      const int e = __shfl_sync(~0u, ent, i & 31);
      valid_bits = e < 0 ? valid_bits & ~(1 << slot) : valid_bits | (1 << slot);
      if (e >= 0) pending |= 1u << slot;
      if (e >= 0 && lane == 0) {
        uint64_t* bar = &full[warp][slot];
        mbar_arrive_expect_tx(bar, C::STAGE);
        tma_load_3d(ring_p + slot * C::STAGE, &kmap, 0, e * PA_BLOCK, 0, bar);
        tma_load_3d(ring_p + slot * C::STAGE + PA_BLOCK * C::ROW, &vmap, 0, e * PA_BLOCK, 0, bar);
      }
    };
#pragma unroll
    for (int k = 0; k < C::STAGES - C::U; ++k) issue(k, k);

    // Q^T fragments: column r of group w is query head 8 w + r of the stream's g,
    // zero past g.  8-bit caches: fp16 and bf16 queries both go to fp16, scaled by
    // a power of two so that the head's largest element lies in [1, 2).
    // sc: scale of the scores of this lane's columns 2 c, 2 c + 1.
    uint32_t qb[NH][C::KS][2];
    float sc[NH][2];
#pragma unroll
    for (int w = 0; w < NH; ++w) {
      const int i = r + 8 * w;
      const bool live = i < p.g;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)b * p.q_sb +
                          (int64_t)(h * p.g + (live ? i : 0)) * p.q_sh;
      if constexpr (E4) {
        // channels 64 i + 16 c + 4 j + {0, 1}, {2, 3} in step 4 i + j
        uint2 v[C::KS];
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
          v[s] = *reinterpret_cast<const uint2*>(q + (s / 4) * 64 + 16 * c + 4 * (s % 4));
        auto get = [&](int s, int k) {
          const uint16_t u = (uint16_t)((k < 2 ? v[s].x : v[s].y) >> (16 * (k % 2)));
          return p.q_bf16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
        };
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(get(s, k)));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        // 2^e <= top < 2^(e+1); a zero, tiny or infinite head is left as it is
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        if (e < -100 || e > 126) e = 0;
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        const float back = __uint_as_float((uint32_t)(127 + e) << 23) * p.scale2 * (p.ks ? p.ks[h] : 1.f);
        sc[w][0] = __shfl_sync(~0u, back, 8 * c);
        sc[w][1] = __shfl_sync(~0u, back, 8 * c + 4);
#pragma unroll
        for (int s = 0; s < C::KS; ++s) {
          const __half2 x = __floats2half2_rn(get(s, 0) * f, get(s, 1) * f);
          const __half2 y = __floats2half2_rn(get(s, 2) * f, get(s, 3) * f);
          qb[w][s][0] = live ? *reinterpret_cast<const uint32_t*>(&x) : 0u;
          qb[w][s][1] = live ? *reinterpret_cast<const uint32_t*>(&y) : 0u;
        }
      } else {
        sc[w][0] = sc[w][1] = p.scale2;
#pragma unroll
        for (int s = 0; s < C::KS; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 * k + 2 * c);
            qb[w][s][k] = live ? v : 0u;
          }
      }
    }

    float o[NH][C::KS][4];                     // O^T: rows channels, columns heads
#pragma unroll
    for (int w = 0; w < NH; ++w)
#pragma unroll
      for (int j = 0; j < C::KS; ++j) o[w][j][0] = o[w][j][1] = o[w][j][2] = o[w][j][3] = 0.f;
    // for each of the lane's heads: reference of the exponents (the largest score so
    // far or a little less), sum over its own tokens, what is added to a scaled score
    // (so large at first that any score moves the reference, and that a masked one
    // still weighs nothing)
    float m[NH][2], l[NH][2], mref[NH][2];
#pragma unroll
    for (int w = 0; w < NH; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) m[w][k] = -CUDART_INF_F, l[w][k] = 0.f, mref[w][k] = PA_UNSET;

    if (p.scores && j0 == 0 && warp == 0 && r == 0) {
      // the scores are kept unscaled
#pragma unroll
      for (int w = 0; w < NH; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (8 * w + 2 * c + k < p.g) p.stat[stream * p.g + 8 * w + 2 * c + k].z = sc[w][k];
    }

    int slot = 0;
    for (int i = 0; i < count && !gave_up; i += C::U) {
      // the slots before these were read in the last step, by all lanes
      __syncwarp();
      const int behind = slot == 0 ? C::STAGES - C::U : slot - C::U;
#pragma unroll
      for (int u = 0; u < C::U; ++u) issue(i + C::STAGES - C::U + u, behind + u);
      int left[C::U];                          // live tokens of a block (16 or more: all)
      float s[C::U][NH][4];                    // S^T: rows tokens tok_r, + 8; columns heads
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        left[u] = 0;
        if (i + u < count && (valid_bits >> (slot + u) & 1)) {
          left[u] = n - (j0 + warp + NW * (i + u)) * PA_BLOCK;
          const bool ok = mbar_wait(&full[warp][slot + u], phases >> (slot + u) & 1);
          if (__all_sync(~0u, ok)) {
            phases ^= 1u << (slot + u);
            pending &= ~(1u << (slot + u));
          } else {
            // the copy stays pending: it is waited for once more below
            if (lane == 0 && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
            gave_up = true;
          }
        }
        // Chains of accumulation, for their latency and because a chain cuts each sum
        // off towards zero.
        constexpr int CH = WIDE ? 2 : 4;
        float part[CH][NH][4];
#pragma unroll
        for (int x = 0; x < CH; ++x)
#pragma unroll
          for (int w = 0; w < NH; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[x][w][k] = 0.f;
        const uint8_t* sk = ring_p + (slot + u) * C::STAGE;
        if constexpr (E4) {
#pragma unroll
          for (int x = 0; x < C::KL; ++x) {
            const uint4 v0 = *reinterpret_cast<const uint4*>(sk + piece_on(k_at, 4 * x));
            const uint4 v1 = *reinterpret_cast<const uint4*>(sk + piece_on(k_at, 4 * x) + 8 * C::SW);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t a[4];
              e4m3x4_to_f16(w0[k], a[0], a[2]);
              e4m3x4_to_f16(w1[k], a[1], a[3]);
#pragma unroll
              for (int w = 0; w < NH; ++w) mma_acc<false>(part[k % CH][w], a, qb[w][4 * x + k][0], qb[w][4 * x + k][1]);
            }
          }
        } else {
          const uint32_t sa = smem_u32(sk);
#pragma unroll
          for (int ks = 0; ks < C::KS; ++ks) {
            uint32_t a[4];
            ldsm4<false>(sa + piece_on(k_at, 2 * ks), a);
#pragma unroll
            for (int w = 0; w < NH; ++w) mma_acc<C::BF16>(part[ks % CH][w], a, qb[w][ks][0], qb[w][ks][1]);
          }
        }
#pragma unroll
        for (int w = 0; w < NH; ++w)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[u][w][k] = part[0][w][k] + part[1][w][k];
            if constexpr (CH == 4) s[u][w][k] += part[2][w][k] + part[3][w][k];
          }
        if (left[u] < PA_BLOCK) {
#pragma unroll
          for (int w = 0; w < NH; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (tok_r + 8 * (k >> 1) >= left[u]) s[u][w][k] = -CUDART_INF_F;
        }
        if (p.scores && i + u < count) {
          // 8 rows of a column are one 32-byte sector
          const int tok0 = (j0 + warp + NW * (i + u)) * PA_BLOCK + tok_r;
#pragma unroll
          for (int w = 0; w < NH; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int head = 8 * w + 2 * c + (k & 1);
              if (head < p.g)
                p.scores[(stream * p.g + head) * p.score_stride + tok0 + 8 * (k >> 1)] = s[u][w][k];
            }
        }
      }
      // The reference m (of the unscaled products: the scale is positive) moves
      // only where a score passes it by more than PA_SLACK, which a lane sees
      // from its own scores: after a few steps that hardly happens, and the
      // lanes' maximum and the scaling of o are skipped.
      bool grows = false;
      float top[NH][2];
#pragma unroll
      for (int w = 0; w < NH; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[w][k] = -CUDART_INF_F;
#pragma unroll
          for (int u = 0; u < C::U; ++u) top[w][k] = fmaxf(top[w][k], fmaxf(s[u][w][k], s[u][w][k + 2]));
          grows |= fmaf(top[w][k], sc[w][k], mref[w][k]) > PA_BIAS + PA_SLACK;
        }
      if (__any_sync(~0u, grows)) {
#pragma unroll
        for (int w = 0; w < NH; ++w) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = top[w][k];
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            x = fmaxf(x, m[w][k]);
            f[k] = x > m[w][k] ? exp2_fast((m[w][k] - x) * sc[w][k]) : 1.f;
            l[w][k] *= f[k];
            m[w][k] = x;
            if (x != -CUDART_INF_F) mref[w][k] = PA_BIAS - __fmul_rn(x, sc[w][k]);   // rounded as in the join
          }
#pragma unroll
          for (int j = 0; j < C::KS; ++j) {
            o[w][j][0] *= f[0], o[w][j][1] *= f[1];
            o[w][j][2] *= f[0], o[w][j][3] *= f[1];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        // P^T: tokens 0..7 and 8..15, high and low parts; two bf16 parts leave 2^-18,
        // which an fp32 output would show, so there a third follows (a variant of its
        // own: a test in the loop costs 1 % at 128K)
        uint32_t ph[NH][2], pl[NH][2], pr[NH][2];
#pragma unroll
        for (int w = 0; w < NH; ++w)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float x = exp2_fast(fmaf(s[u][w][2 * t], sc[w][0], mref[w][0]));
            const float y = exp2_fast(fmaf(s[u][w][2 * t + 1], sc[w][1], mref[w][1]));
            l[w][0] += x;
            l[w][1] += y;
            split_pair<C::BF16>(x, y, ph[w][t], pl[w][t], pr[w][t]);
            ph[w][t] = transpose8(ph[w][t]);
            pl[w][t] = transpose8(pl[w][t]);
            if constexpr (THIRD) pr[w][t] = transpose8(pr[w][t]);
          }
        // The products cut their sums off towards zero, which over many blocks adds
        // up (2e-5 after 400): a block's are summed by themselves and added to O
        // with rounding to nearest.
        auto pv = [&](int j, const uint32_t (&a)[4]) {
#pragma unroll
          for (int w = 0; w < NH; ++w) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (THIRD) mma_acc<C::BF16>(t, a, pr[w][0], pr[w][1]);
            mma_acc<C::BF16>(t, a, pl[w][0], pl[w][1]);
            mma_acc<C::BF16>(t, a, ph[w][0], ph[w][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[w][j][k] += t[k];
          }
        };
        const uint8_t* sv = ring_p + (slot + u) * C::STAGE + PA_BLOCK * C::ROW;
        const bool part = left[u] < PA_BLOCK;  // what lies behind the sequence in its last page may be anything
        if constexpr (E4) {
#pragma unroll
          for (int x = 0; x < C::VL; ++x) {
            uint32_t v[4][C::VB / 4];          // tokens 2 c, (2 c + 1) ^ 4, and 8 further
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint8_t* from = sv + piece_on(t & 1 ? v_at1 : v_at, 8 * x) + (t >> 1) * 8 * C::SW;
              if constexpr (C::VB == 16) {
                const uint4 y = *reinterpret_cast<const uint4*>(from);
                v[t][0] = y.x, v[t][1] = y.y, v[t][2] = y.z, v[t][3] = y.w;
              } else {
                const uint2 y = *reinterpret_cast<const uint2*>(from);
                v[t][0] = y.x, v[t][1] = y.y;
              }
            }
            if (part) {
#pragma unroll
              for (int t = 0; t < 4; ++t)
                if (8 * (t >> 1) + ((t & 1) ? (2 * c + 1) ^ 4 : 2 * c) >= left[u]) {
#pragma unroll
                  for (int y = 0; y < C::VB / 4; ++y) v[t][y] = 0u;
                }
            }
#pragma unroll
            for (int y = 0; y < C::VB / 4; ++y) {
              uint32_t a[4], d[4];
              e4m3x4_to_f16(__byte_perm(v[0][y], v[1][y], 0x5140), a[0], a[1]);
              e4m3x4_to_f16(__byte_perm(v[2][y], v[3][y], 0x5140), a[2], a[3]);
              pv(x * (C::VB / 2) + 2 * y, a);
              e4m3x4_to_f16(__byte_perm(v[0][y], v[1][y], 0x7362), d[0], d[1]);
              e4m3x4_to_f16(__byte_perm(v[2][y], v[3][y], 0x7362), d[2], d[3]);
              pv(x * (C::VB / 2) + 2 * y + 1, d);
            }
          }
        } else {
          const uint32_t sa = smem_u32(sv);
#pragma unroll
          for (int j = 0; j < C::KS; ++j) {
            uint32_t a[4];
            ldsm4<true>(sa + piece_on(v_at, 2 * j), a);
            if (part) {
              // pairs of tokens 2 c, 2 c + 1 and 8 further
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const int tok = 2 * c + 8 * (t >> 1);
                a[t] &= (tok < left[u] ? 0xffffu : 0u) | (tok + 1 < left[u] ? 0xffff0000u : 0u);
              }
            }
            pv(j, a);
          }
        }
      }
      slot = slot + C::U == C::STAGES ? 0 : slot + C::U;
    }
    // the reference in the scaled domain from here on
#pragma unroll
    for (int w = 0; w < NH; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) m[w][k] = m[w][k] == -CUDART_INF_F ? m[w][k] : __fmul_rn(m[w][k], sc[w][k]);

    if (gave_up) {
      // copies in flight must have landed before the ring is used for anything else
      for (int k = 0; k < C::STAGES; ++k)
        if (pending >> k & 1) mbar_wait(&full[warp][k], phases >> k & 1);
      pending = 0;
    }
    // join the warps: the ring is drained and becomes [warp][head][D + 4]
#pragma unroll
    for (int w = 0; w < NH; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = l[w][k];
        x += __shfl_xor_sync(~0u, x, 4);
        x += __shfl_xor_sync(~0u, x, 8);
        x += __shfl_xor_sync(~0u, x, 16);
        if (r == 0) sm_m[warp][8 * w + 2 * c + k] = m[w][k], sm_l[warp][8 * w + 2 * c + k] = x;
      }
    __syncthreads();
    float* mg = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int w = 0; w < NH; ++w)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int head = 8 * w + 2 * c + k;
        float top = sm_m[0][head];
#pragma unroll
        for (int x = 1; x < NW; ++x) top = fmaxf(top, sm_m[x][head]);
        // a part without a live token stays zero
        const bool none = m[w][k] == -CUDART_INF_F;
        const float f = none ? 0.f : exp2f(m[w][k] - top);
        float* to = mg + (warp * C::HR + head) * (D + 4);
#pragma unroll
        for (int j = 0; j < C::KS; ++j) {
          const float x = none ? 0.f : o[w][j][k] * f, y = none ? 0.f : o[w][j][2 + k] * f;
          if constexpr (E4) {
            // tile j: channels 2 j, 2 j + 1 of the lane's piece
            constexpr int T = C::VB / 2;       // tiles of a piece
            *reinterpret_cast<float2*>(to + (j / T) * 8 * C::VB + C::VB * r + 2 * (j % T)) = make_float2(x, y);
          } else {
            to[16 * j + r] = x;
            to[16 * j + 8 + r] = y;
          }
        }
      }
    __syncthreads();
    const bool whole = j0 == 0 && j1 == nb && p.cluster == 1;
    float* own = reinterpret_cast<float*>(smem + C::MERGE);
    const float vs = CT == MKV_DT_E4M3 && p.vs ? p.vs[h] : 1.f;
    const int64_t part = 2 * (int64_t)blockIdx.x + (j0 == 0 ? 1 : 0);
    for (int e = tid; e < p.g * (D / 4); e += NW * 32) {
      const int head = e / (D / 4), d = (e - head * (D / 4)) * 4;
      float top = sm_m[0][head];
#pragma unroll
      for (int k = 1; k < NW; ++k) top = fmaxf(top, sm_m[k][head]);
      float sum = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float mk = sm_m[k][head];
        sum += mk == -CUDART_INF_F ? sm_l[k][head] : sm_l[k][head] * exp2f(mk - top);
        const float4 v = *reinterpret_cast<const float4*>(mg + (k * C::HR + head) * (D + 4) + d);
        a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
      }
      a.x *= vs, a.y *= vs, a.z *= vs, a.w *= vs;
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t row = stream * p.g + head;
        store_out4(p, row * D + d, a, inv);
        if (d == 0) {
          store_stat(p, row, top, sum);
        }
      } else if (!p.split) {
        *reinterpret_cast<float4*>(own + head * D + d) = a;
        if (d == 0) own_ml[head] = make_float2(top, sum);
      } else {
        *reinterpret_cast<float4*>(p.part_o + (part * p.g + head) * D + d) = a;
        if (d == 0) {
          p.part_ml[(part * p.g + head) * 2] = top;
          p.part_ml[(part * p.g + head) * 2 + 1] = sum;
        }
      }
    }
    if (!p.split) {
      if (p.cluster > 1) {
        // the ranks' sums, joined over distributed shared memory: each rank an even
        // share of the elements
        namespace cg = cooperative_groups;
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        for (int e = (int)cl.block_rank() * NW * 32 + tid; e < p.g * (D / 4); e += p.cluster * NW * 32) {
          const int head = e / (D / 4), d = (e - head * (D / 4)) * 4;
          float2 ml[8];
          float4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < p.cluster) {
              ml[q] = *cl.map_shared_rank(&own_ml[head], q);
              v[q] = *reinterpret_cast<const float4*>(cl.map_shared_rank(own + head * D + d, q));
            }
          float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < p.cluster) top = fmaxf(top, ml[q].x);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < p.cluster) {
              const float f = ml[q].x == top ? 1.f : exp2f(ml[q].x - top);
              sum += ml[q].y * f;
              a.x += v[q].x * f, a.y += v[q].y * f, a.z += v[q].z * f, a.w += v[q].w * f;
            }
          const int64_t row = stream * p.g + head;
          store_out4(p, row * D + d, a, sum == 0.f ? 0.f : 1.f / sum);
          if (d == 0) store_stat(p, row, top, sum);
        }
        cl.sync();                    // no rank's sums are read any more
      }
      break;
    }
    if (at < g1) {                  // the merge area becomes the ring again
      fence_proxy_async();
      __syncthreads();
    }
  }
}

template <int CT, int D, bool WIDE, int NW, bool THIRD>
cudaError_t launch_pa_third(const PagedAttnParams& p, cudaStream_t st) {
  using C = PA<CT, D, WIDE, NW>;
  CUtensorMap kmap, vmap;
  if (cudaError_t e = encode_rows_map(&kmap, p.kp, p.rows, C::ROW, PA_BLOCK)) return e;
  if (cudaError_t e = encode_rows_map(&vmap, p.vp, p.rows, C::ROW, PA_BLOCK)) return e;
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<CT, D, WIDE, NW, THIRD>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = p.split ? PA_SHARES * p.G : (int64_t)p.B * p.H * p.cluster;
  return launch_kernel(paged_attn_kernel<CT, D, WIDE, NW, THIRD>, dim3((unsigned)grid), dim3(NW * 32), C::SMEM, st, true, p.cluster,
                       p, kmap, vmap);
}

template <int CT, int D, bool WIDE, int NW>
cudaError_t launch_pa_nw(const PagedAttnParams& p, cudaStream_t st) {
  if constexpr (CT == MKV_DT_BF16)
    if (p.out_type == MKV_DT_F32) return launch_pa_third<CT, D, WIDE, NW, true>(p, st);
  return launch_pa_third<CT, D, WIDE, NW, false>(p, st);
}

// 4 warps a CTA and several CTAs an SM; where all CTAs run at once with one an SM
// (of 152 SMs clusters of 8 reach about half), 8 warps.  Rows of 512 bytes, whose
// rings do not fit, apart.
template <int CT, int D, bool WIDE>
cudaError_t launch_pa(const PagedAttnParams& p, cudaStream_t st) {
  if constexpr (PA<CT, D, WIDE, 4>::ROW < 512)
    if ((p.split ? p.G : (int64_t)p.B * p.H * p.cluster) <= (p.cluster == 8 ? p.sms / 2 : p.sms))
      return launch_pa_nw<CT, D, WIDE, 8>(p, st);
  return launch_pa_nw<CT, D, WIDE, 4>(p, st);
}

template <int D>
cudaError_t launch_pa_d(const PagedAttnParams& p, int cache_type, cudaStream_t st) {
  const bool wide = p.g > 8;
  switch (cache_type) {
    case MKV_DT_F16: return wide ? launch_pa<MKV_DT_F16, D, true>(p, st) : launch_pa<MKV_DT_F16, D, false>(p, st);
    case MKV_DT_BF16: return wide ? launch_pa<MKV_DT_BF16, D, true>(p, st) : launch_pa<MKV_DT_BF16, D, false>(p, st);
    default: return wide ? launch_pa<MKV_DT_E4M3, D, true>(p, st) : launch_pa<MKV_DT_E4M3, D, false>(p, st);
  }
}

}  // namespace
}  // namespace mkv
