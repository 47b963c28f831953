// Attention of many queries over keys in tensors or in pages on the fifth-generation
// tensor cores, included by one translation unit per head dimension.
//
//   z_ij = score(q_i, k_j) over the keys j that query i sees, o_i = softmax(z_i) v
//
// in one pass over the keys with a running reference m_i of the exponents and sum
// l_i.  The g query heads of a KV head share its keys: a row tile is 128 / g tokens
// times g heads, so that few tokens still fill the 128 rows of a product and the
// keys of a group are read once.
//
// A CTA holds one row tile and walks over blocks of 128 keys (D = 256: 64), or two and
// blocks of 64 (tensor memory has no room for more):
//   S = Q K^T       tcgen05, both operands in shared memory, S in tensor memory;
//   softmax         a warpgroup per row tile, one row a thread (no shuffles): scores
//                   out of tensor memory, exponents, 16-bit weights back over them;
//   O += P V        tcgen05, P in tensor memory, V in shared memory, O in tensor
//                   memory (fp32).
// Roles: one warp copies (TMA, 128-byte swizzle, a ring of K and V tiles), one lane a row
// tile issues its products, a warpgroup a row tile does its softmax.  Every row tile has
// two S buffers: the scores of the block after next are formed while a softmax runs, so
// that none waits for products of its own.  The products of a buffer are issued in the
// order S, P V, next S by one thread, which is the order they execute in.
//
// What bounds it: the tensor cores' pipe, occupied 82 % of the time at 8192 tokens x 4 of 32
// heads over 8, causal, 66 % with arithmetic and the rest with reading operands: 1520 us in
// calls in a row (1425 for one launch by itself, at the clock that a short run has), 1.45
// PFLOP/s of the products that are needed (a library product of large matrices: 1.89);
// without the causal mask, whose blocks on the diagonal are half idle, 1.61.  With two row
// tiles a CTA one softmax runs beside the other's products: of calls in a row 1549 us with
// two S buffers a tile, 2520 with one and an issuing lane for both.
// A short prompt is bound by what a CTA does before its first product and after its last,
// some 8000 cycles, and by its longest row tile: one prompt of 2048 tokens 35 us, 1.9 times
// the products' time.  (Two CTAs an SM with a row tile each, whose starts and ends overlap:
// the same 35 us, and before biased scores were walked from the last key down 72 instead of 62
// for a ragged batch of them; 128 registers a thread are too few.)  Capped or biased scores: by
// the softmax, 4096 x 2 tokens 292 and 243 us for 207.
//
// O is scaled down only where a row's maximum passes its reference by 2^6 (bf16: 2^24):
// after the first blocks that hardly happens, and no work on O lies between the products.
// Weights carry a factor 2^8, which cancels: fp16 ones stay normal down to 2^-22 of
// the largest, and below 2^14.  The rounding of the weights to 16 bits is half a step
// of the output's own type; their sum is of the unrounded ones.
//
// Few rows of a KV head: with 32 or fewer, four copies of them fill the 128 rows, one for
// the lanes of tensor memory of each softmax warp, and a warp takes a quarter of a block's
// columns, with weights of zero in the others; with up to 64 over 8-bit pages, two copies
// and halves (16 drafts of 4 heads over 32 streams of 32768 slots: 111 us, 138 without;
// 16-bit pages: no gain).  A block's softmax is then as much shorter, where otherwise some
// warps would work and the others wait; the copies' parts are joined at the end.
//
// 8-bit pages: a further warpgroup widens the raw tiles to fp16 between the copies and
// the products.
#pragma once

#include <math_constants.h>

#include <algorithm>
#include <cstring>

#include "attend_internal.cuh"
#include "decode_common.cuh"
#include "ptx.cuh"
#include "tc05.cuh"

namespace mkv {
namespace {

enum { FROM_TENSORS = 0, FROM_PAGES = 1, FROM_BYTES = 2 };

template <int D, int TILES, int FROM, int COPIES>
struct AT {
  static constexpr int NB = attend_block(D, TILES, FROM == FROM_BYTES, COPIES > 1);
  static constexpr bool E4 = FROM == FROM_BYTES;
  static constexpr bool FEW = COPIES > 1;
  static constexpr int G = D / 64;                         // groups of 64 channels
  static constexpr int QTILE = 128 * D * 2;
  static constexpr int TILE = NB * D * 2;                  // bytes of a K or V tile
  static constexpr int RAW = NB * D;
  // tiles of the ring: what shared memory holds
  static constexpr int STAGES = E4 ? (D == 64 ? 8 : D == 128 ? 6 : 3) * (D < 256 ? 64 : NB) / NB
                                : D == 256 ? 5
                                : D == 128 ? (TILES == 2 ? 10 : 6)
                                           : (TILES == 2 ? 12 : 8);
  static constexpr int RAWS = E4 ? (D == 256 ? 3 : FEW ? 5 : 8) : 1;
  // columns of a block that a softmax warp takes, and rows of a row tile that are not copies
  static constexpr int COLS = NB / COPIES, ROWS = 128 / COPIES;
  static constexpr int SMEM = TILES * QTILE + STAGES * TILE + (E4 ? RAWS * RAW : 0) + 1024;
  static constexpr int THREADS = TILES == 2 || E4 ? 384 : 256;
  static constexpr int O_COL = TILES * 2 * NB;             // tensor memory columns: S buffers, then O
  static_assert(O_COL + TILES * D <= 512, "tensor memory");
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory");
  static_assert(!FEW || 128 * (D + 4) * 4 + 1024 <= STAGES * TILE + (E4 ? RAWS * RAW : 0), "the join's area");
  static_assert(!(E4 && TILES == 2), "the second warpgroup widens");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// cap2 tanh(a x): x times a polynomial in x^2 with the smallest largest relative error
// (found by exchange), the factors in its coefficients: of degree 4 for |a x| <= 1/2
// (3e-8), of 6 up to 1 (7e-8), both within 3 u of it with their roundings, and without the
// two slow functions of the other form.  16K tokens in documents, capped at 50: 840 us with
// that form alone, 647 with degree 6, 548 with both.
template <int N>
struct SmallTanh {
  float c[N];
  // factor: a cap2
  __device__ __forceinline__ SmallTanh(const float (&of)[N], float a, float factor) {
    float f = factor;
#pragma unroll
    for (int i = 0; i < N; ++i, f *= a * a) c[i] = of[i] * f;
  }
  __device__ __forceinline__ float2 operator()(float2 x) const {
    const float2 u = mul2(x, x);
    float2 y = fma2(u, twice(c[N - 1]), twice(c[N - 2]));
#pragma unroll
    for (int i = N - 3; i >= 0; --i) y = fma2(u, y, twice(c[i]));
    return mul2(x, y);
  }
};
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0u;
}
// Operand descriptors, 128-byte swizzled, version 1: the upper word (rows of 8 1024
// bytes apart) is the same for all, the lower one has the address / 16 and the distance
// of groups of 64 channels / 16 (V, whose channels are contiguous; else not used).
constexpr uint32_t DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) { return (saddr >> 4) | (lead >> 4) << 16; }
// D[tmem] (+)= A B, A and B in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(DESC_HI)
      : "memory");
}
// D[tmem] (+)= A[tmem] B
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "n"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
               "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float* v) {
  if constexpr (N == 32) tmem_ld32(taddr, v);
  else tmem_ld16(taddr, reinterpret_cast<uint32_t*>(v));
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* u) {
  if constexpr (N == 32) tmem_st32(taddr, u);
  else if constexpr (N == 16) tmem_st16(taddr, u);
  else tmem_st8(taddr, u);
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(uint32_t src, const CUtensorMap* map, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
               : "memory");
}
// Until this thread's stores have read the shared memory.
__device__ __forceinline__ void tma_store_read() {
  asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;\n" ::: "memory");
}

// mbar_wait without a call.
__device__ __forceinline__ bool wait_here(uint64_t* bar, uint32_t parity) {
  uint64_t since = 0;
  for (int i = 0; !mbar_test(bar, parity); ++i) {
    if (i < 4096) continue;
    const uint64_t now = globaltimer_ns();
    if (i == 4096) since = now;
    if (now - since > WAIT_LIMIT_NS) return false;
    i = 4096 + 1;
  }
  return true;
}

// The blocks of keys that a CTA walks over, the same in every role (a warp asks as a
// whole): all of a range, or those in which some document of its queries occurs.  DOWN: the
// last first, for scores biased by distance, which are largest there: the exponents'
// reference is near its final value from the start and outputs are rarely scaled (4096 x 2
// tokens 243 us, 302 upwards; without a bias, heads of 256 take 239, 219 upwards: CTAs that
// start together then read the same keys).
template <bool DOWN>
struct Blocks {
  int j, end, base;      // left are [j, end)
  uint32_t bits;         // of the 32 blocks from base on (which may be below 0): taken;
  uint32_t lone;         // of one document alone, `doc`
  int doc;
  const int2* range;     // of the sequence's blocks; NULL: all
  int2 own;              // of the queries' documents
  __device__ __forceinline__ uint32_t hits(int from, uint32_t& one) const {
    const int i = from + (int)(threadIdx.x & 31);
    bool hit = false, same = false;
    if (i >= j && i < end) {
      const int2 r = range[i];
      hit = r.x <= own.y && r.y >= own.x;
      same = r.x == doc && r.y == doc;
    }
    one = __ballot_sync(~0u, same);
    return __ballot_sync(~0u, hit);
  }
  // block i, the last that next() gave, has nothing but `doc`
  __device__ __forceinline__ bool plain(int i) const { return lone >> (i - base) & 1; }
  // before the walk: (how many, the highest)
  __device__ __forceinline__ int2 all() const {
    if (!range) return make_int2(max(0, end - j), end - 1);
    int2 r = make_int2(0, -1);
    for (int from = j; from < end; from += 32) {
      uint32_t one;
      const uint32_t h = hits(from, one);
      r.x += __popc(h);
      if (h) r.y = from + 31 - __clz(h);
    }
    return r;
  }
  __device__ __forceinline__ int next() {
    if (!range) return j < end ? DOWN ? --end : j++ : -1;
    while (j < end) {
      if (DOWN ? end <= base : j >= base + 32) {
        base = DOWN ? end - 32 : j;
        bits = hits(base, lone);
      }
      const uint32_t rest = DOWN ? bits & (~0u >> (32 - (end - base))) : bits >> (j - base);
      if (rest) {
        if (DOWN) return end = base + 31 - __clz(rest);
        j += __ffs(rest);
        return j - 1;
      }
      if (DOWN) end = base;
      else j = base + 32;
    }
    return -1;
  }
};

// Bits of the columns [lo, hi) of a block among the 32 from `first` on.
__device__ __forceinline__ uint32_t columns(int lo, int hi, int first) {
  const int a = max(lo - first, 0), b = min(hi - first, 32);
  return a >= b ? 0u : (~0u << a) & (~0u >> (32 - b));
}

struct AttendShared {
  uint64_t q_full;
  uint64_t full[12], empty[12];        // K and V tiles as the products take them
  uint64_t raw_full[8], raw_empty[8];  // 8-bit tiles
  uint64_t s_full[4], p_full[4];       // a buffer's scores are there; its weights are
  uint64_t o_last[2];                  // all products of a row tile are in O
  uint64_t o_ready[2];                 // its output is in shared memory
  uint32_t tmem;
  int depth[64];                       // of a tree's new tokens
  uint32_t absent[16];                 // pages: of the last 16 blocks, units whose page is not in the cache
  float q_scale[128];                  // 8-bit pages: what a row of q was divided by
  uint64_t joins[2];                   // few rows: references and sums are there; outputs
};

// ---------------------------------------------------------------------------
// grid: B * H * groups * splits; block AT::THREADS; dynamic smem AT::SMEM
// ---------------------------------------------------------------------------
template <int D, int TILES, int FROM, bool BF16, int MODS, int COPIES>
__global__ void __launch_bounds__(AT<D, TILES, FROM, COPIES>::THREADS, 1)
    attend_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap omap, int unit) {
  using C = AT<D, TILES, FROM, COPIES>;
  constexpr int NB = C::NB, G = C::G;
  constexpr bool CAP = (MODS & 1) != 0, SLOPES = (MODS & 2) != 0;      // scores are capped, biased
  constexpr bool FOLDS = MODS == 0;        // see AT_FOLD
  constexpr bool E4 = C::E4, PAGED = FROM != FROM_TENSORS, FEW = C::FEW;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttendShared sh;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem_p = smem_raw + (smem0 - smem_u32(smem_raw));
  const uint32_t ring = smem0 + TILES * C::QTILE, raws = ring + C::STAGES * C::TILE;
  // the same for a warp, and known to be: addresses and descriptors stay in uniform registers
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);

  if (warp == 1) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 0) {
    if (lane < 12) {
      mbar_init(&sh.full[lane], E4 ? 4 : 1);
      mbar_init(&sh.empty[lane], TILES);
    } else if (lane < 20) {
      mbar_init(&sh.raw_full[lane - 12], 1);
      mbar_init(&sh.raw_empty[lane - 12], 4);
    } else if (lane < 24) {
      mbar_init(&sh.s_full[lane - 20], 1);
      mbar_init(&sh.p_full[lane - 20], 4);
    } else if (lane < 26) {
      mbar_init(&sh.o_last[lane - 24], 1);
      mbar_init(&sh.o_ready[lane - 24], 4);
    } else if (lane == 26) {
      mbar_init(&sh.q_full, E4 ? 4 : 1);
    } else if (lane < 29) {
      mbar_init(&sh.joins[lane - 27], 4);
    }
    mbar_init_fence();
  }
  griddep_wait();

  // this CTA's part: row tiles [tile0, tile0 + TILES) of (b, h), the part-th share of their keys
  // (in bundles of (sequence, KV head) pairs, whose keys several CTAs then read at the same
  // time; of a bundle, what may see the most keys first)
  int rest = blockIdx.x, streams = p.B * p.H, bh = 0;
  if (streams > AT_BUNDLE) {
    const int size = AT_BUNDLE * p.groups * p.splits, bundle = rest / size;
    bh = bundle * AT_BUNDLE;
    streams = min(streams - bh, AT_BUNDLE);
    rest -= bundle * size;
  }
  const int width = streams * p.splits, of = rest / width;
  rest -= of * width;
  const int stream = p.splits > 1 ? rest / p.splits : rest, part = rest - stream * p.splits;
  bh += stream;
  const int group = p.groups - 1 - of, b = bh / p.H, h = bh - b * p.H;
  const int64_t cta = ((int64_t)bh * p.groups + of) * p.splits + part;    // its place in the workspace
  const int TT = p.tile_tokens, t0 = group * TILES * TT;
  int m, L;
  bool outside;
  attend_lens(p, b, m, L, outside);
  if (outside && PAGED && p.status && h == 0 && group == 0 && part == 0 && tid == 0) atomicOr(p.status, DEV_ERR_CHECK);
  const int base = L - m;
  const int t1 = min(m, t0 + TILES * TT);                // tokens of this CTA: [t0, t1)
  const int prefix = p.prefix ? p.prefix[b] : 0;
  // keys that a token at place `at` sees, as a range
  auto first_key = [&](int at) { return p.window ? (int)max((int64_t)0, (int64_t)at - p.window + 1) : 0; };
  auto end_key = [&](int at) {
    if (p.causal) return min(L, max(at + 1, prefix));
    return p.window ? (int)min((int64_t)L, (int64_t)at + p.window) : L;
  };
  int lo = 0, hi = 0;
  if (t0 < t1) {
    lo = first_key(base + t0);
    hi = end_key(base + t1 - 1);
    if (p.tree) lo = first_key(base), hi = L;
  }
  const int32_t* docs = p.docs ? p.docs + b * p.docs_stride : nullptr;
  Blocks<SLOPES> blocks;
  blocks.range = nullptr;
  blocks.doc = 0;
  {
    const int from = lo / NB, n = hi > lo ? (hi + NB - 1) / NB - from : 0;
    blocks.j = from;
    blocks.end = from + n;
    if (p.splits > 1) {                // n * splits fits 32 bits: 2^24 blocks, 64 parts
      blocks.j = from + (uint32_t)n * part / (uint32_t)p.splits;
      blocks.end = from + (uint32_t)n * (part + 1) / (uint32_t)p.splits;
    }
    blocks.base = SLOPES ? blocks.end : blocks.j - 32;
  }
  if (docs && hi > lo) {
    int2 own = make_int2(INT32_MAX, INT32_MIN);
    for (int t = t0 + lane; t < t1; t += 32)
      if (base + t >= 0) {
        const int d = docs[base + t];
        own.x = min(own.x, d), own.y = max(own.y, d);
      }
    blocks.own.x = __reduce_min_sync(~0u, own.x);
    blocks.own.y = __reduce_max_sync(~0u, own.y);
    blocks.range = p.doc_range + (int64_t)b * ((p.nk + NB - 1) / NB);
  }
  if (p.tree && tid < m) {
    const uint64_t valid = m >= 64 ? ~0ull : (1ull << m) - 1;
    sh.depth[tid] = __popcll(p.tree[(int64_t)b * p.nq + tid] & valid & ~(1ull << tid));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a kernel behind this one may take tensor memory before it waits for this one,
  // which all of this grid has by then
  griddep_launch();
  const uint32_t tmem = __shfl_sync(~0u, sh.tmem, 0);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(~0u, wait_here(bar, parity));
    if (!ok && lane == 0 && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
    return ok;
  };

  if (warp < 4) {
    if (warp == 0) {
      // ---- copies -----------------------------------------------------------
      const bool work = blocks.all().x > 0;
      if constexpr (!E4) {
        if (work) {
          constexpr int TIMES = FEW ? COPIES : TILES;
          if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, TIMES * G * TT * p.g * 128);
          __syncwarp();
          if (lane < TIMES * G) {
            const int i = lane / G, c = lane - i * G;
            tma_load_4d(smem0 + c * 128 * 128 + i * (FEW ? C::ROWS * 128 : C::QTILE), &qmap, c * 64, h * p.g,
                        t0 + (FEW ? 0 : i * TT), b, &sh.q_full);
          }
        }
      }
      uint64_t* const full = E4 ? sh.raw_full : sh.full;
      uint64_t* const empty = E4 ? sh.raw_empty : sh.empty;
      constexpr int SLOTS = E4 ? C::RAWS : C::STAGES, BYTES = E4 ? C::RAW : C::TILE;
      const uint32_t at0 = E4 ? raws : ring;
      int n = 0, slot = 0;
      uint32_t turn = 0;
      bool ok = true;
      // pages: this lane's unit of the 32 from `from` (which may be below 0) on, and bits of those whose page is not
      // in the cache; apart for keys and values, which are two blocks behind
      struct Units {
        int from = SLOPES ? INT32_MAX : INT32_MIN, entry = 0;
        uint32_t gone = 0;
      } key_units, value_units;
      int step = 0;
      const int per = NB / unit;
      auto load = [&](const CUtensorMap& map, int j, bool keys) {
        if (!ok) return;
        if (n >= SLOTS && !(ok = wait(&empty[slot], (turn & 1) ^ 1))) return;
        const uint32_t at = at0 + slot * BYTES;
        if constexpr (PAGED) {
          const int u0 = j * per;
          Units& units = keys ? key_units : value_units;
          if (SLOPES ? u0 < units.from : u0 - 32 >= units.from) {
            units.from = SLOPES ? u0 + per - 32 : u0;
            const int t = (units.from + lane) * unit;
            int entry = p.n_pages * p.H * p.page_size;     // behind the pool: zeros
            bool bad = false;
            if (t >= 0 && t < L) {
              const int pg = t / p.page_size;
              const int page = p.table[b * p.table_stride + pg];
              bad = page < 0 || page >= p.n_pages;
              if (!bad) entry = (page * p.H + h) * p.page_size + (t - pg * p.page_size);
            }
            units.entry = entry;
            units.gone = __ballot_sync(~0u, bad);
          }
          const uint32_t lost = (units.gone >> (u0 - units.from)) & ((1u << per) - 1);
          if (lane == 0) {
            if (lost && p.status) atomicOr(p.status, DEV_ERR_CHECK);
            // read by the softmax behind this block's scores, so behind this copy's arrival
            if (keys) sh.absent[step & 15] = lost;
            mbar_arrive_expect_tx(&full[slot], BYTES);
          }
          if (keys) ++step;
          constexpr int W = E4 ? 1 : G;
          const int u = lane / W, c = lane - u * W;
          const int row = __shfl_sync(~0u, units.entry, (u0 - units.from + u) & 31);
          __syncwarp();
          if (u < per) tma_load_2d(at + c * NB * 128 + u * unit * (E4 ? D : 128), &map, c * 64, row, &full[slot]);
        } else {
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], BYTES);
          __syncwarp();
          if (lane < G) tma_load_4d(at + lane * NB * 128, &map, lane * 64, j * NB, h, b, &full[slot]);
        }
        ++n;
        if (++slot == SLOTS) slot = 0, ++turn;
      };
      int cur = blocks.next();
      if (cur >= 0) load(kmap, cur, true);
      int nxt = cur >= 0 ? blocks.next() : -1;
      if (nxt >= 0) load(kmap, nxt, true);
      while (cur >= 0 && ok) {
        const int then = nxt >= 0 ? blocks.next() : -1;
        load(vmap, cur, false);
        if (then >= 0) load(kmap, then, true);
        cur = nxt;
        nxt = then;
      }
      // no copy may be in flight when the CTA ends
      for (int i = max(0, n - SLOTS); i < n; ++i) wait_here(&full[i % SLOTS], (i / SLOTS) & 1);
      if (!E4 && work) wait_here(&sh.q_full, 0);
    } else if (warp <= TILES) {
      // ---- products ---------------------------------------------------------
      // One lane of a warp does it all for a row tile: between two products there is room
      // for some hundred cycles, and while one tile's lane waits the other's products run.
      constexpr uint32_t IS = idesc_f16_f32(128, NB) | (BF16 && !E4 ? (1u << 7) | (1u << 10) : 0u);
      constexpr uint32_t IO = idesc_f16_f32(128, D) | (BF16 && !E4 ? (1u << 7) | (1u << 10) : 0u) | (1u << 16);
      const int tile = warp - 1;
      const int2 all = blocks.all();
      const int n = all.x;
      const bool leader = elect_one();
      const uint32_t s0 = tmem + 2 * tile * NB, o0 = tmem + C::O_COL + tile * D;
      const uint32_t qa = desc_lo(smem0 + tile * C::QTILE, 16);
      int slot = 0;
      uint32_t turn = 0;
      bool ok = true;
      auto pop = [&]() {       // the next tile of the ring, once it is there
        const int s = slot;
        ok = ok && wait_here(&sh.full[s], turn & 1);
        if (++slot == C::STAGES) slot = 0, ++turn;
        return s;
      };
      // scores of block k into buffer k mod 2, and the product with its weights
      auto scores = [&](int k) {
        const int s = pop();
        if (!ok) return;
        tc_fence_after();
        const uint32_t ka = desc_lo(ring + s * C::TILE, 16);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          mma_ss(s0 + (k & 1) * NB, qa + ((c / 4) * 128 * 128 + (c % 4) * 32) / 16,
                 ka + ((c / 4) * NB * 128 + (c % 4) * 32) / 16, IS, c > 0);
        tc_commit(&sh.s_full[2 * tile + (k & 1)]);
        tc_commit(&sh.empty[s]);
      };
      auto values = [&](int k) {
        const int s = pop();
        ok = ok && wait_here(&sh.p_full[2 * tile + (k & 1)], (k >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t va = desc_lo(ring + s * C::TILE, NB * 128);
#pragma unroll
        for (int c = 0; c < NB / 16; ++c)
          mma_ts(o0, s0 + (k & 1) * NB + c * 8, va + c * 2048 / 16, IO, (FOLDS ? (k & p.fold) != 0 : k > 0) || c > 0);
        tc_commit(&sh.empty[s]);
      };
      // What lies behind the sequence in its last block may be anything, and 0 times a
      // NaN is one: those rows of V become zeros (8-bit pages: where they are widened).
      // It is the last tile of V (DOWN: the first); of two warps both write the zeros they need.
      auto clean = [&](int j) {
        const int at_n = SLOPES ? min(n, 2) : 2 * n - 1, s = at_n % C::STAGES;
        wait_here(&sh.full[s], (at_n / C::STAGES) & 1);
        uint8_t* at = smem_p + TILES * C::QTILE + s * C::TILE;
        const int r0 = L - j * NB;
        for (int i = lane; i < (NB - r0) * 8; i += 32) {
#pragma unroll
          for (int c = 0; c < G; ++c)
            *reinterpret_cast<uint4*>(at + c * NB * 128 + (r0 + i / 8) * 128 + (i % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      };
      if (leader && n > 0) {
        ok = wait_here(&sh.q_full, 0);
        scores(0);
        if (n > 1) scores(1);
        for (int k = 0; !SLOPES && k + 1 < n && ok; ++k) {
          values(k);
          if (k + 2 < n) scores(k + 2);
        }
      }
      __syncwarp();
      if (!E4 && n > 0 && (all.y + 1) * NB > L) clean(all.y);
      __syncwarp();
      if (leader && n > 0) {
        for (int k = SLOPES ? 0 : n - 1; k < n && ok; ++k) {
          values(k);
          if (SLOPES && k + 2 < n) scores(k + 2);
        }
        tc_commit(&sh.o_last[tile]);
        if (!ok && p.status) atomicOr(p.status, DEV_ERR_TIMEOUT);
        // no product may be in flight when the tensor memory goes
        wait_here(&sh.o_last[tile], 0);
      }
    }
  } else if (!E4 || warp < 8) {
    // ---- softmax: a row a thread --------------------------------------------
    const int tile = TILES == 2 ? (warp >> 2) - 1 : 0;
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int rt = row % C::ROWS / p.g, head = h * p.g + (row % C::ROWS - rt * p.g);
    const int token = t0 + tile * TT + rt;
    const bool live = rt < TT && token < t1;
    const int copy = row / C::ROWS, col0 = copy * C::COLS;   // which rows these are a copy of; its columns of a block
    const bool any = __any_sync(~0u, live);
    // what this row sees: keys [klo, khi), of its document, and the new tokens of its tree row
    int place = base + token, klo = 0, khi = INT32_MAX;
    uint64_t sees = 0;
    if (live) {
      if (p.tree) {
        const uint64_t valid = m >= 64 ? ~0ull : (1ull << m) - 1;
        sees = p.tree[(int64_t)b * p.nq + token] & valid;
        place = base + sh.depth[token];
        klo = first_key(place);
        khi = base;
        if (p.window)
          for (int j = 0; j < m; ++j)
            if (sh.depth[token] - sh.depth[j] >= p.window) sees &= ~(1ull << j);
      } else {
        klo = first_key(place);
        khi = end_key(place);
        if (docs && place < 0) khi = 0;
      }
    }
    const int doc = docs && live && place >= 0 ? docs[place] : 0;
    // blocks [whole0, whole1): all keys seen by all rows of the warp (but for their documents)
    const int whole0 = ((int)__reduce_max_sync(~0u, live ? klo : 0) + NB - 1) / NB;
    const int whole1 = (int)__reduce_min_sync(~0u, khi) / NB;
    // all rows of the warp of one document: its blocks are known 32 at a time
    blocks.doc = __reduce_max_sync(~0u, live ? doc : INT32_MIN);
    const bool one_doc = __all_sync(~0u, !live || doc == blocks.doc);
    // the first of the warp's places
    const int nearest = MODS ? (int)__reduce_min_sync(~0u, live ? place : INT32_MAX) : 0;
    float sc = p.scale * 1.4426950408889634f;            // of the products, to log2
    const float slope = SLOPES && live ? p.slopes[head] * 1.4426950408889634f : 0.f;
    bool ok = true;
    if (E4 && blocks.j < blocks.end) {
      ok = wait(&sh.q_full, 0);
      sc *= sh.q_scale[row] * (p.k_scale ? p.k_scale[h] : 1.f);
    }
    {
      // products to the tanh's argument; for caps so small that the polynomials' factors would
      // overflow infinite, which sends all scores to the exact form
      float into = CAP ? sc / (p.cap * 1.4426950408889634f) : 0.f;
      if constexpr (CAP) {
        const float f = into * into * into;
        if (!(sc * f * f * f * f <= 1e30f)) into = CUDART_INF_F;
      }
      const SmallTanh<5> small({1.f, -0.3333306908607483f, 0.13324779272079468f, -0.05298607423901558f, 0.017135007306933403f},
                               into, sc);
      const float by = MODS ? 1.f : sc;
      float top = -CUDART_INF_F, mref = 1e38f, l = 0.f;
      constexpr int COLS = C::COLS, W = COLS < 32 ? COLS : 32;   // columns at a time
      uint32_t k = 0;
      const uint32_t o_at = tmem + lanes + C::O_COL + tile * D;
      for (int j = ok ? blocks.next() : -1; j >= 0; j = blocks.next(), ++k) {
        const int buf = 2 * tile + (k & 1);
        const uint32_t w_at = tmem + lanes + buf * NB, s_at = w_at + col0;
        if (!(ok = wait(&sh.s_full[buf], (k >> 1) & 1))) break;
        if (any) {
          tc_fence_after();
          const int j0 = j * NB + col0;
          // columns that some row does not see
          bool masked = j < whole0 || j >= whole1;
          uint32_t absent = 0;
          if constexpr (PAGED) {
            absent = sh.absent[k & 15];
            masked |= absent != 0;
          }
          int2 dr = make_int2(doc, doc);
          if (docs && !(one_doc && blocks.plain(j))) {
            dr = blocks.range[j];
            masked |= __any_sync(~0u, live && (dr.x != doc || dr.y != doc));
          }
          // bits of the 32 columns from c0 on that this row sees
          auto seen = [&](int c0) {
            const int k0 = j0 + c0;
            uint32_t bits = live ? columns(klo, khi, k0) : 0u;
            if (p.tree) {
              const int off = k0 - base;
              bits |= off >= 0 ? (off < 64 ? (uint32_t)(sees >> off) : 0u) : off > -32 ? (uint32_t)sees << -off : 0u;
            }
            if (docs) {
              if (dr.x == dr.y) {
                bits = dr.x == doc ? bits : 0u;
              } else if (__any_sync(~0u, bits != 0u)) {
                uint32_t same = 0;
                for (int i = 0; i < 32; ++i)
                  if (k0 + i < L && docs[k0 + i] == doc) same |= 1u << i;
                bits &= same;
              }
            }
            if (PAGED && absent)
              for (int i = 0; i < 32; i += 16)
                if (absent >> ((col0 + c0 + i) / unit) & 1) bits &= ~(0xffffu << i);
            return bits;
          };
          if (!MODS && masked) {
            // in tensor memory, 32 at a time: beside the pass below it would cost plain blocks
            // registers (8K prompts, batch 4: 1645 us instead of 1549)
#pragma unroll 1
            for (int c0 = 0; c0 < COLS; c0 += 32) {
              float v[W];
              tmem_load<W>(s_at + c0, v);
              tmem_ld_wait();
              const uint32_t bits = seen(c0);
#pragma unroll
              for (int i = 0; i < W; ++i)
                if (!(bits >> i & 1)) v[i] = -CUDART_INF_F;
              tmem_store<W>(s_at + c0, reinterpret_cast<const uint32_t*>(v));
            }
            tmem_st_wait();
          }
          float v[COLS];
#pragma unroll
          for (int c = 0; c < COLS; c += W) tmem_load<W>(s_at + c, v + c);
          tmem_ld_wait();
          if constexpr (MODS != 0) {
            if constexpr (CAP) {
              float large[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int c = 0; c < COLS; c += 2) large[c / 2 % 4] = max3(large[c / 2 % 4], fabsf(v[c]), fabsf(v[c + 1]));
              const float big = live ? fmaxf(max3(large[0], large[1], large[2]), large[3]) : 0.f;
              // The form goes by the scores that rows which are there see: forms differ in their
              // roundings, and the rest may be anything.  What the other forms need is hidden from
              // the compiler until there: taken out of the loop over the blocks it costs this one
              // its registers (4096 x 2 tokens: 316 us, 292).
              if (__all_sync(~0u, big * into <= 0.5f)) {
#pragma unroll
                for (int i = 0; i < COLS; i += 2) {
                  const float2 y = small(make_float2(v[i], v[i + 1]));
                  v[i] = y.x, v[i + 1] = y.y;
                }
              } else if (E4 || masked) {
                float a = into, top2 = p.cap, by1 = sc;
                asm volatile("" : "+f"(a), "+f"(top2), "+f"(by1));
                top2 *= 1.4426950408889634f;
                // some score is larger, perhaps one that is not seen: W at a time.  8-bit pages' kernels,
                // which have the fewest registers, know no other way (64 drafts over 4 streams of
                // 65536 slots of 64: 271 us, 231).
#pragma unroll 1
                for (int c0 = 0; c0 < COLS; c0 += W) {
                  const uint32_t bits = masked ? seen(c0) : live ? ~0u : 0u;
                  float t[W];
                  tmem_load<W>(s_at + c0, t);
                  tmem_ld_wait();
                  float most[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                  for (int i = 0; i < W; ++i)
                    if (bits >> i & 1) most[i % 4] = fmaxf(most[i % 4], fabsf(t[i]));
                  const float arg = fmaxf(max3(most[0], most[1], most[2]), most[3]) * a;
                  if (__all_sync(~0u, arg <= 0.5f)) {
#pragma unroll
                    for (int i = 0; i < W; i += 2) {
                      const float2 y = small(make_float2(t[i], t[i + 1]));
                      t[i] = y.x, t[i + 1] = y.y;
                    }
                  } else {
                    const CappedScore capped(top2);
                    if (top2 <= 128.f) {
                      const float to2 = fminf(by1 / top2 * 2.885390081777927f, 3.402823466e38f);
#pragma unroll
                      for (int i = 0; i < W; ++i) t[i] = capped.large(t[i] * to2);
                    } else {
#pragma unroll
                      for (int i = 0; i < W; ++i) t[i] = capped(t[i] * by1);
                    }
                  }
                  tmem_store<W>(s_at + c0, reinterpret_cast<const uint32_t*>(t));
                }
                tmem_st_wait();
#pragma unroll
                for (int c = 0; c < COLS; c += W) tmem_load<W>(s_at + c, v + c);
                tmem_ld_wait();
              } else if (__all_sync(~0u, big * into <= 1.f)) {
                float a = into, by1 = sc;
                asm volatile("" : "+f"(a), "+f"(by1));
                const SmallTanh<7> medium({0.9999999403953552f, -0.33332839608192444f, 0.13325203955173492f,
                                           -0.05345702916383743f, 0.020289979875087738f, -0.006203379016369581f,
                                           0.0010410225950181484f},
                                          a, by1);
#pragma unroll
                for (int i = 0; i < COLS; i += 2) {
                  const float2 y = medium(make_float2(v[i], v[i + 1]));
                  v[i] = y.x, v[i + 1] = y.y;
                }
              } else {
                float top2 = p.cap, by1 = sc;
                asm volatile("" : "+f"(top2), "+f"(by1));
                top2 *= 1.4426950408889634f;
                const CappedScore capped(top2);
                if (top2 <= 128.f) {     // an error of 2^-22 of so small a cap is less than the products'
                  const float to2 = fminf(by1 / top2 * 2.885390081777927f, 3.402823466e38f);
#pragma unroll
                  for (int i = 0; i < COLS; ++i) v[i] = capped.large(v[i] * to2);
                } else {
#pragma unroll
                  for (int i = 0; i < COLS; ++i) v[i] = capped(v[i] * by1);
                }
              }
            } else if (j0 + COLS <= nearest + 1 && !(p.tree && j0 + COLS > base)) {
              // all keys before all rows: the distance is linear
              const float2 sc2 = twice(sc), slope2 = twice(slope), off2 = twice(-slope * (float)(place - j0));
#pragma unroll
              for (int c = 0; c < COLS; c += 2) {
                const float2 y = fma2(make_float2(v[c], v[c + 1]), sc2, fma2(slope2, make_float2((float)c, (float)(c + 1)), off2));
                v[c] = y.x, v[c + 1] = y.y;
              }
            } else {
#pragma unroll
              for (int c = 0; c < COLS; ++c) v[c] *= sc;
            }
            if (SLOPES && (CAP || j0 + COLS > nearest + 1 || (p.tree && j0 + COLS > base))) {
              const float far = (float)(place - j0);
              if (p.tree && j0 + NB > base) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                  const int t = j0 + c - base;
                  v[c] -= slope * fabsf(t < 0 ? far - (float)c : (float)(place - base - sh.depth[min(t, 63)]));
                }
              } else {
#pragma unroll
                for (int c = 0; c < COLS; ++c) v[c] -= slope * fabsf(far - (float)c);
              }
            }
            if (masked) {
#pragma unroll
              for (int c0 = 0; c0 < COLS; c0 += 32) {
                const uint32_t bits = seen(c0);
#pragma unroll
                for (int i = 0; i < W; ++i)
                  if (!(bits >> i & 1)) v[c0 + i] = -CUDART_INF_F;
              }
            }
          }
          float x = fmaxf(v[0], v[1]), x1 = fmaxf(v[2], v[3]);
#pragma unroll
          for (int c = 4; c < COLS; c += 4) {
            x = max3(x, v[c], v[c + 1]);
            x1 = max3(x1, v[c + 2], v[c + 3]);
          }
          x = fmaxf(x, x1);
          const bool grows = live && fmaf(x, by, mref) > AT_BIAS + (BF16 && !E4 ? AT_SLACK_BF16 : AT_SLACK);
          const bool folds = FOLDS && (k & p.fold) == 0 && k > 0;
          if (__any_sync(~0u, grows) || folds) {
            float f = 1.f;
            if (grows) {
              if (top != -CUDART_INF_F) f = ex2((top - x) * by);
              top = x;
              l *= f;
              mref = AT_BIAS - __fmul_rn(x, by);
            }
            if (k > 0) {
              // O by the same factor, between its products: the last one has run when its V tile
              // (the ring's 2 k-th, or the one before where there is but one block) is released
              const int used = 2 * k;
              if (!(ok = wait(&sh.empty[used % C::STAGES], (used / C::STAGES) & 1))) break;
              tc_fence_after();
              const bool held = FOLDS && (int)k - 1 > p.fold;       // some are in the workspace
              if (folds || held) {
                int at = row;
                asm volatile("" : "+r"(at));               // addressed here: outside the loop it costs registers
                float4* kept = p.part_o + (cta * TILES + tile) * (D / 4) * 128 + at;
#pragma unroll 1
                for (int c = 0; c < D; c += 16, kept += 4 * 128) {
                  uint32_t o[16];
                  tmem_ld16(o_at + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    float4 w = held ? kept[i * 128] : make_float4(0.f, 0.f, 0.f, 0.f);
                    if (folds) {
                      w.x += __uint_as_float(o[4 * i]), w.y += __uint_as_float(o[4 * i + 1]);
                      w.z += __uint_as_float(o[4 * i + 2]), w.w += __uint_as_float(o[4 * i + 3]);
                    }
                    kept[i * 128] = make_float4(w.x * f, w.y * f, w.z * f, w.w * f);
                  }
                }
              }
#pragma unroll
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_at + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(o_at + c, o);
              }
            }
          }
          float2 s0 = make_float2(0.f, 0.f), s1 = s0;
          const float2 by2 = twice(by), mref2 = twice(mref);
#pragma unroll
          for (int c0 = 0; c0 < COLS; c0 += W) {
            uint32_t w[W / 2];
#pragma unroll
            for (int c = 0; c < W; c += 4) {
              float2 a = fma2(make_float2(v[c0 + c], v[c0 + c + 1]), by2, mref2);
              float2 d = fma2(make_float2(v[c0 + c + 2], v[c0 + c + 3]), by2, mref2);
              a = make_float2(ex2(a.x), ex2(a.y));
              d = make_float2(ex2(d.x), ex2(d.y));
              s0 = add2(s0, a);
              s1 = add2(s1, d);
              w[c / 2] = pack16<(BF16 && !E4)>(a.x, a.y);
              w[c / 2 + 1] = pack16<(BF16 && !E4)>(d.x, d.y);
            }
            tmem_store<W / 2>(w_at + (col0 + c0) / 2, w);
          }
          if constexpr (FEW) {
            // the other copies' keys weigh nothing in this one
            uint32_t none[W / 2];
#pragma unroll
            for (int i = 0; i < W / 2; ++i) none[i] = 0u;
#pragma unroll
            for (int i = COLS; i < NB; i += W) tmem_store<W / 2>(w_at + (col0 + i) % NB / 2, none);
          }
          s0 = add2(s0, s1);
          l += s0.x + s0.y;
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[buf]);
      }
      // ---- this row's result --------------------------------------------------
      // (with copies of the rows every warp has its part in the join)
      const bool joins = FEW ? t0 < t1 : any;
      if (ok && joins && k > 0) ok = wait(&sh.o_last[tile], 0);
      // 32 channels of the row's sums, those in the workspace among them
      auto sums = [&](int c, float (&o)[32]) {
        tmem_ld32(o_at + c, o);
        tmem_ld_wait();
        if (FOLDS && (int)k - 1 > p.fold) {
          const float4* kept = p.part_o + ((cta * TILES + tile) * (D / 4) + c / 4) * 128 + row;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 w = kept[i * 128];
            o[4 * i] += w.x, o[4 * i + 1] += w.y, o[4 * i + 2] += w.z, o[4 * i + 3] += w.w;
          }
        }
      };
      // A row tile without padding goes out by one copy, through the shared memory of its
      // queries, which no product needs any more; otherwise every thread writes its row.
      const bool whole = !FEW && p.splits == 1 && t0 + (tile + 1) * TT <= t1;
      if (FEW && ok && joins) {
        // few rows: the copies' parts of each, over a common reference, by way of the shared
        // memory of K and V
        tc_fence_after();
        constexpr int LD = D + 4;
        float* all = reinterpret_cast<float*>(smem_p + C::QTILE);
        float2* few_ml = reinterpret_cast<float2*>(all + 128 * LD);    // [copy][row]
        const float vscale = E4 && p.v_scale ? p.v_scale[h] : 1.f;
        few_ml[row] = make_float2(top == -CUDART_INF_F ? top : __fmul_rn(top, by), l);
        auto meet = [&](int i) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.joins[i]);
          return wait(&sh.joins[i], 0);
        };
        ok = meet(0);
        auto joined = [&](int r, float2& ml) {       // (reference, sum) of row r
          ml = few_ml[r];
#pragma unroll
          for (int q = 1; q < COPIES; ++q) ml.x = fmaxf(ml.x, few_ml[q * C::ROWS + r].x);
          ml.y = 0.f;
#pragma unroll
          for (int q = 0; q < COPIES; ++q) {
            const float2 x = few_ml[q * C::ROWS + r];
            ml.y += x.x == -CUDART_INF_F ? x.y : x.y * ex2(x.x - ml.x);
          }
        };
        float2 ml;
        joined(row % C::ROWS, ml);
        const float mine = few_ml[row].x;
        const float f = mine == -CUDART_INF_F ? 0.f : ex2(mine - ml.x) * vscale;
        float* to = all + row * LD;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (k > 0) sums(c, o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(to + c + 4 * i) =
                l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[4 * i] * f, o[4 * i + 1] * f, o[4 * i + 2] * f, o[4 * i + 3] * f);
        }
        ok = ok && meet(1);
        const int rows = (t1 - t0) * p.g;
        for (int e = row; ok && e < rows * (D / 4); e += 128) {
          const int r = e / (D / 4), c = (e - r * (D / 4)) * 4;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int q = 0; q < COPIES; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(all + (q * C::ROWS + r) * LD + c);
            a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
          }
          joined(r, ml);
          const int tk = t0 + r / p.g, hd = h * p.g + r % p.g;
          if (p.splits > 1) {
            p.part_o[(cta * (D / 4) + c / 4) * 128 + r] = a;
            if (c == 0) p.part_ml[cta * 128 + r] = ml;
          } else {
            const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
            uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.os[0] + (int64_t)tk * p.os[1] + hd * p.os[2] + c;
            *reinterpret_cast<uint2*>(out) = make_uint2(pack16<BF16>(a.x * inv, a.y * inv), pack16<BF16>(a.z * inv, a.w * inv));
            if (c == 0 && p.lse)
              p.lse[((int64_t)b * p.nq + tk) * p.Hq + hd] =
                  ml.y == 0.f ? -CUDART_INF_F : (ml.x + (log2f(ml.y) - AT_BIAS)) * 0.6931471805599453f;
          }
        }
      } else if (ok && any) {
        tc_fence_after();
        const float vscale = E4 && p.v_scale ? p.v_scale[h] : 1.f;
        const float mine = top == -CUDART_INF_F ? top : __fmul_rn(top, by);
        const int64_t part_row = (cta * TILES + tile) * 128 + row;
        const float inv = p.splits > 1 ? vscale : l > 0.f ? vscale / l : l == 0.f ? 0.f : l;   // a NaN stays one
        uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.os[0] + (int64_t)token * p.os[1] + head * p.os[2];
        if (live) {
          if (p.splits > 1) p.part_ml[part_row] = make_float2(mine, l);
          else if (p.lse)
            p.lse[((int64_t)b * p.nq + token) * p.Hq + head] =
                l == 0.f ? -CUDART_INF_F : (mine + (log2f(l) - AT_BIAS)) * 0.6931471805599453f;
        }
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (k > 0) sums(c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
          if (p.splits > 1) {
            float4* to = p.part_o + ((cta * TILES + tile) * (D / 4) + c / 4) * 128 + row;
            if (live) {
#pragma unroll
              for (int i = 0; i < 8; ++i) to[i * 128] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 u;
              u.x = pack16<BF16>(o[8 * i], o[8 * i + 1]);
              u.y = pack16<BF16>(o[8 * i + 2], o[8 * i + 3]);
              u.z = pack16<BF16>(o[8 * i + 4], o[8 * i + 5]);
              u.w = pack16<BF16>(o[8 * i + 6], o[8 * i + 7]);
              if (whole)
                *reinterpret_cast<uint4*>(smem_p + tile * C::QTILE + (c / 64) * 128 * 128 + row * 128 +
                                          (((c / 8 + i) & 7) ^ (row & 7)) * 16) = u;
              else if (live)
                *reinterpret_cast<uint4*>(out + c + 8 * i) = u;
            }
          }
        }
      }
      if (ok && whole) {
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_ready[tile]);
        if ((warp & 3) == 0 && wait(&sh.o_ready[tile], 0) && lane < G) {
          tma_store_4d(smem0 + tile * C::QTILE + lane * 128 * 128, &omap, lane * 64, h * p.g, t0 + tile * TT, b);
          tma_store_read();
        }
        __syncwarp();
      }
    }
  } else if constexpr (E4) {
    // ---- widening: 8-bit tiles to fp16 ----------------------------------------
    const int row = tid & 127;
    if (blocks.j < blocks.end) {
      // queries: fp16 and bf16 both go to fp16, a row scaled by a power of two so that its
      // largest element lies in [1, 2)
      const int rt = row % C::ROWS / p.g, head = h * p.g + (row % C::ROWS - rt * p.g), token = t0 + rt;
      const bool live = rt < TT && token < t1;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.qs[0] + (int64_t)(live ? token : 0) * p.qs[1] +
                          (live ? head : 0) * p.qs[2];
      auto get = [&](uint32_t w, int i) {
        const uint16_t u = (uint16_t)(w >> (16 * i));
        return BF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
      };
      float big = 0.f;
      if (live)
        for (int c = 0; c < D; c += 8) {
          const uint4 u = *reinterpret_cast<const uint4*>(q + c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(get(w[i / 2], i % 2)));
        }
      int e = (int)(__float_as_uint(big) >> 23) - 127;
      if (e < -100 || e > 126) e = 0;                    // zero, tiny or infinite: as it is
      const float f = __uint_as_float((uint32_t)(127 - e) << 23);
      sh.q_scale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
      for (int c = 0; c < D; c += 8) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (live) {
          u = *reinterpret_cast<const uint4*>(q + c);
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack16<false>(get(w[i], 0) * f, get(w[i], 1) * f);
          u = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(smem_p + (c / 64) * 128 * 128 + row * 128 + (((c / 8) & 7) ^ (row & 7)) * 16) = u;
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    }
    int n = 0;
    bool ok = true;
    auto widen = [&](int j, bool values) {
      if (!ok) return;
      const int rs = n % C::RAWS, s = n % C::STAGES;
      if (!(ok = wait(&sh.raw_full[rs], (n / C::RAWS) & 1))) return;
      if (n >= C::STAGES && !(ok = wait(&sh.empty[s], (n / C::STAGES - 1) & 1))) return;
      // a thread takes the same 16 channels of every RS-th row: a multiple of 8 rows, so that
      // the swizzle is the same for all
      constexpr int PIECES = D / 16, RS = 128 / PIECES;
      const int r0 = row / PIECES, c = row % PIECES, ch = (2 * c) & 7;
      const uint8_t* from = smem_p + C::QTILE + C::STAGES * C::TILE + rs * C::RAW + row * 16;
      uint8_t* to = smem_p + C::QTILE + s * C::TILE + (c / 4) * NB * 128 + r0 * 128;
      uint8_t *to0 = to + ((ch ^ (r0 & 7)) << 4), *to1 = to + (((ch + 1) ^ (r0 & 7)) << 4);
      const int keep = values ? L - j * NB : NB;        // rows behind the sequence become zeros
#pragma unroll
      for (int i = 0; i < NB / RS; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(from + i * 128 * 16);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[8];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
              : "=r"(o[2 * x]), "=r"(o[2 * x + 1])
              : "r"(w[x]));
        if (r0 + i * RS >= keep) {
#pragma unroll
          for (int x = 0; x < 8; ++x) o[x] = 0u;
        }
        *reinterpret_cast<uint4*>(to0 + i * RS * 128) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(to1 + i * RS * 128) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.raw_empty[rs]);
        mbar_arrive(&sh.full[s]);
      }
      ++n;
    };
    int cur = blocks.next();
    if (cur >= 0) widen(cur, false);
    int nxt = cur >= 0 ? blocks.next() : -1;
    if (nxt >= 0) widen(nxt, false);
    while (cur >= 0 && ok) {
      const int then = nxt >= 0 ? blocks.next() : -1;
      widen(cur, true);
      if (then >= 0) widen(then, false);
      cur = nxt;
      nxt = then;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int TILES, int FROM, bool BF16, int MODS, int COPIES>
cudaError_t launch_at(const AttendParams& p, cudaStream_t st) {
  using C = AT<D, TILES, FROM, COPIES>;
  CUtensorMap qmap, kmap, vmap, omap;
  std::memset(&qmap, 0, sizeof(qmap));
  int unit = C::NB;
  // the stride of an extent of 1 is never walked, but has to be one that a map takes
  auto walked = [](int64_t stride, int64_t extent) { return (uint64_t)(extent > 1 ? stride * 2 : 16); };
  if constexpr (FROM == FROM_TENSORS) {
    const uint32_t box[4] = {64, (uint32_t)C::NB, 1, 1};
    const uint64_t dim[4] = {(uint64_t)D, (uint64_t)std::max(p.nk, 1), (uint64_t)p.H, (uint64_t)p.B};
    for (int i = 0; i < 2; ++i) {
      const int64_t* s = i ? p.vs : p.ks;
      const uint64_t stride[3] = {walked(s[1], p.nk), walked(s[2], p.H), walked(s[0], p.B)};
      if (cudaError_t e = encode_map(i ? &vmap : &kmap, p.nk ? (i ? p.v : p.k) : p.q, false, 4, dim, stride, box, true)) return e;
    }
  } else {
    int a = p.page_size, r = C::NB;
    while (r) {
      const int t = a % r;
      a = r, r = t;
    }
    unit = a;
    const uint64_t dim[2] = {(uint64_t)D, (uint64_t)p.n_pages * p.H * p.page_size};
    const uint64_t stride[1] = {(uint64_t)D * (C::E4 ? 1 : 2)};
    const uint32_t box[2] = {C::E4 ? (uint32_t)D : 64u, (uint32_t)unit};
    for (int i = 0; i < 2; ++i)
      if (cudaError_t e = encode_map(i ? &vmap : &kmap, i ? p.v : p.k, C::E4, 2, dim, stride, box, !C::E4)) return e;
  }
  for (int i = C::E4 ? 1 : 0; i < 2; ++i) {
    const int64_t* s = i ? p.os : p.qs;
    const uint64_t dim[4] = {(uint64_t)D, (uint64_t)p.Hq, (uint64_t)p.nq, (uint64_t)p.B};
    const uint64_t stride[3] = {walked(s[2], p.Hq), walked(s[1], p.nq), walked(s[0], p.B)};
    const uint32_t box[4] = {64, (uint32_t)p.g, (uint32_t)p.tile_tokens, 1};
    if (cudaError_t e = encode_map(i ? &omap : &qmap, i ? p.out : p.q, false, 4, dim, stride, box, true)) return e;
  }
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, TILES, FROM, BF16, MODS, COPIES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_kernel(attend_kernel<D, TILES, FROM, BF16, MODS, COPIES>, dim3((unsigned)((int64_t)p.B * p.H * p.groups * p.splits)), dim3(C::THREADS),
                       C::SMEM, st, true, 0, p, qmap, kmap, vmap, omap, unit);
}

// Scores that are capped or biased are a kernel of their own: their code would cost the
// plain one registers.
template <int D, int TILES, int FROM, int COPIES>
cudaError_t launch_options(const AttendParams& p, cudaStream_t st) {
  const int mods = (p.cap > 0.f ? 1 : 0) | (p.slopes ? 2 : 0);
  switch (mods) {
    case 0: return p.bf16 ? launch_at<D, TILES, FROM, true, 0, COPIES>(p, st) : launch_at<D, TILES, FROM, false, 0, COPIES>(p, st);
    case 1: return p.bf16 ? launch_at<D, TILES, FROM, true, 1, COPIES>(p, st) : launch_at<D, TILES, FROM, false, 1, COPIES>(p, st);
    case 2: return p.bf16 ? launch_at<D, TILES, FROM, true, 2, COPIES>(p, st) : launch_at<D, TILES, FROM, false, 2, COPIES>(p, st);
    default: return p.bf16 ? launch_at<D, TILES, FROM, true, 3, COPIES>(p, st) : launch_at<D, TILES, FROM, false, 3, COPIES>(p, st);
  }
}

template <int D, int TILES, int COPIES>
cudaError_t launch_from(const AttendParams& p, cudaStream_t st) {
  if (!p.table) return launch_options<D, TILES, FROM_TENSORS, COPIES>(p, st);
  if (p.cache_type != MKV_DT_E4M3) return launch_options<D, TILES, FROM_PAGES, COPIES>(p, st);
  if constexpr (TILES == 1) return launch_options<D, 1, FROM_BYTES, COPIES>(p, st);
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_attend_d(const AttendParams& p, cudaStream_t st) {
  if constexpr (D < 256)
    if (p.tiles == 2) return launch_from<D, 2, 1>(p, st);
  return launch_from<D, 1, 1>(p, st);
}

}  // namespace
}  // namespace mkv
