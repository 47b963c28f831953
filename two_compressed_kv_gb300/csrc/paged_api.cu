// Host side of the rotary and paged-cache calls in include/mkv.h: argument
// checks, workspace layout and launch order.  No state is kept between calls.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include <cudaTypedefs.h>

#include "paged_internal.cuh"

using namespace mkv;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int64_t kMaxGrid = 0x7fffffff;

#define CKP(call)                                              \
  do {                                                         \
    cudaError_t e_ = (call);                                   \
    if (e_ != cudaSuccess) return set_cuda_error(e_, #call);   \
  } while (0)

mkv_status bad(const char* text) { return set_error(MKV_ERR_INVALID_ARG, text); }

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is16(int dtype) { return dtype == MKV_DT_F16 || dtype == MKV_DT_BF16; }
// Stride of a dimension that is walked over: 16-byte accesses need multiples of 8
// elements.  That of an extent of 1 is never used.
bool stride8(int64_t stride, int64_t extent) { return extent <= 1 || stride % 8 == 0; }
int elem_bytes(int dtype) { return dtype == MKV_DT_F32 ? 4 : dtype == MKV_DT_E4M3 ? 1 : 2; }

// SMs of the current device.
mkv_status sm_count(int* out) {
  int dev = 0;
  CKP(cudaGetDevice(&dev));
  CKP(cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev));
  return MKV_OK;
}

// Heads a thread takes so that its angles serve several heads while the grid
// still has at least `want` threads: a 32K prefill of 8 heads takes 170, 100, 83
// and 81 us with 1, 2, 4 and 8, one step of 8 x 32 heads 2.4 us with 1, 3.5 with 8.
int heads_per_thread(int64_t threads, int heads, int64_t want, int most) {
  int per = 1;
  while (per < most && per < heads && threads * up(heads, 2 * per) >= want) per *= 2;
  return std::min(per, heads);
}

const char* check_plan(const mkv_rope_plan* p) {
  if (p->head_dim < 1 || p->head_dim > 4096 || p->rot_dim < 2 || p->rot_dim % 2 != 0 ||
      p->rot_dim > p->head_dim || p->rot_dim > 2 * MKV_ROPE_MAX_PAIRS || p->interleaved < 0 ||
      p->interleaved > 1 || !std::isfinite(p->mult))
    return "the rope plan was not made by mkv_rope_plan_init";
  return nullptr;
}

const char* check_cache(const mkv_paged_cache* c) {
  if (!c) return "paged cache: NULL view";
  if (!c->k_pages || !c->v_pages || !c->page_table) return "paged cache: NULL pages or page table";
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages)) return "paged cache: pages must be 16-byte aligned";
  if (c->dtype != MKV_DT_F16 && c->dtype != MKV_DT_BF16 && c->dtype != MKV_DT_E4M3)
    return "paged cache: dtype must be F16, BF16 or E4M3";
  if ((c->k_scale || c->v_scale) && c->dtype != MKV_DT_E4M3) return "paged cache: scales are for E4M3 only";
  if (c->batch < 1 || c->batch > 65535) return "paged cache: batch must be 1..65535";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535) return "paged cache: n_kv_heads must be 1..65535";
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return "paged cache: head_dim must be 64, 128 or 256";
  if (c->page_size < 16 || c->page_size > 256 || c->page_size % 16 != 0)
    return "paged cache: page_size must be a multiple of 16 from 16 to 256";
  if (c->n_pages < 1 || c->max_pages < 1) return "paged cache: n_pages and max_pages must be >= 1";
  if ((int64_t)c->max_pages * c->page_size > ((int64_t)1 << 30))
    return "paged cache: max_pages * page_size must be <= 2^30";
  if (c->table_stride < c->max_pages) return "paged cache: table_stride must be >= max_pages";
  if ((int64_t)c->n_pages * c->n_kv_heads > kMaxGrid / c->page_size)
    return "paged cache: too many pages (n_pages * n_kv_heads * page_size must be below 2^31)";
  return nullptr;
}

// ---- decode ------------------------------------------------------------------

// Up to this many tokens a CTA, a cluster of CTAs takes each stream and joins its
// parts over distributed shared memory; beyond, or with more sequences than fit
// the split kernel's prefix sums, the load is split over all streams and a second
// kernel joins.  Us of clusters and of the split, group 4, D = 128, equal lengths:
//   8 streams    1024: 6.4, 9.9    4096: 8.8, 11.8   16384: 19.2, 20.8
//   32 streams   1024: 7.2, 11.3   4096: 15.9, 20.2   8192: 26.1, 30.4
//   64 streams   1024: 9.8, 17.1   4096: 25.9, 33.5
//   256 streams  1024: 24.6, 36.7  2048: 44.0, 56.0
// Lengths are not known to the host, and one long sequence among short ones takes
// as long as its own CTAs: 64 x 4 streams, one of 16384 tokens: 52 us in clusters
// of 4, 20 split; spread up to 16384: 96 and 76 us.  So the bound is low.
constexpr int64_t kClusterTokens = 2048;

// CTAs of a stream: as many as run at once for all streams (clusters of 8: 16 of
// them do not: 16 streams of 4096 take 17.2 us with 8, 12.5 with 4), each with 64
// tokens or more of the bound (8 streams of 304: 6.3 us with 1, 5.9 with 2, 5.6 with 4).
int stream_cluster(int64_t streams, int64_t limit) {
  int n = streams <= 8 ? 8 : streams <= 32 ? 4 : streams <= 64 ? 2 : 1;
  while (n > 1 && limit < 64 * n) n /= 2;
  return n;
}

// Smallest share of a CTA of the split kernel: 8 blocks of 16 tokens.
constexpr int kMinBlocks = 8;

// What a part of a stream costs a CTA apart from its blocks (its queries, the
// first copies' latency, the join of the warps), in blocks.  256 ragged e4m3
// streams: 76.3 us with 32, 81.8 with 8; equal long streams: no difference.
constexpr int kPieceLoad = 32;
// Sixteenths of the load handed out in small shares, from so many blocks a CTA
// on.  With 0, 2 and 4: the ragged batch 90.6, 80.9 and 76.3 us, fp16 32K batch 4
// 93.4, 92.1 and 88.4, 128K batch 8 633, 603 and 607.
constexpr int kTail16 = 4;
constexpr int kTailFrom = 64;

struct DecodeLayout {
  bool split;
  int cluster, G;
  int64_t limit;
  int64_t score_stride;
  uint64_t part_o, part_ml, stat, pre, scores, total;   // byte offsets
};

const char* check_decode(const mkv_paged_cache* c, const mkv_paged_decode_args* a) {
  if (const char* e = check_cache(c)) return e;
  if (!a) return "mkv_paged_decode: NULL arguments";
  if (a->n_q_heads < 1 || a->n_q_heads % c->n_kv_heads != 0)
    return "mkv_paged_decode: n_q_heads must be a multiple of n_kv_heads";
  if (a->n_q_heads / c->n_kv_heads > MAX_G) return "mkv_paged_decode: at most 16 query heads per KV head";
  if (!is16(a->q_dtype) || (c->dtype != MKV_DT_E4M3 && a->q_dtype != c->dtype))
    return "mkv_paged_decode: q must be F16 or BF16, of the cache's type unless that is E4M3";
  if (a->out_dtype != a->q_dtype && a->out_dtype != MKV_DT_F32)
    return "mkv_paged_decode: out must be of q's type or F32";
  if (a->max_len < 0 || a->max_len > (int64_t)c->max_pages * c->page_size)
    return "mkv_paged_decode: max_len must be 0..max_pages * page_size";
  if (!(a->scale >= 0.f) || std::isinf(a->scale)) return "mkv_paged_decode: scale must be >= 0 and finite";
  if ((int64_t)c->batch * a->n_q_heads > kMaxGrid) return "mkv_paged_decode: too many heads";
  return nullptr;
}

int64_t decode_limit(const mkv_paged_cache* c, const mkv_paged_decode_args* a) {
  const int64_t cap = (int64_t)c->max_pages * c->page_size;
  return a->max_len ? std::min(a->max_len, cap) : cap;
}

DecodeLayout decode_layout(const mkv_paged_cache* c, const mkv_paged_decode_args* a, int sms) {
  DecodeLayout l;
  const int64_t g = a->n_q_heads / c->n_kv_heads;
  const int64_t streams = (int64_t)c->batch * c->n_kv_heads;
  l.limit = decode_limit(c, a);
  l.cluster = stream_cluster(streams, l.limit);
  l.split = l.limit > kClusterTokens * l.cluster && c->batch <= PA_MAX_B;
  if (l.split) l.cluster = 1;
  // Large shares for two CTAs an SM at most: a third slot, where there is one, then
  // takes small shares all the time (256 ragged e4m3 streams 79.6 -> 75.3 us, 32 of
  // 32768 61.0 -> 56.7; 16 heads: 32 e4m3 streams of 65536 141 -> 131.5, 256 ragged
  // ones 119.5 -> 110.6, 32 fp16 streams of 65536 in rows of 64 105.5 -> 98.0).
  const int ctas = std::min(2, paged_ctas(c->head_dim * elem_bytes(c->dtype)));
  l.G = (int)std::min<int64_t>((int64_t)sms * ctas,
                               streams * up(up(l.limit, PA_BLOCK), kMinBlocks));
  l.score_stride = up(l.limit, 16) * 16;
  uint64_t at = 0;
  auto place = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) & ~(uint64_t)255;
    return here;
  };
  l.part_o = place(l.split ? 2ull * PA_SHARES * l.G * g * c->head_dim * 4 : 0);
  l.part_ml = place(l.split ? 2ull * PA_SHARES * l.G * g * 8 : 0);
  l.pre = place(l.split ? 8ull * (c->batch + 1) : 0);
  l.stat = place((uint64_t)streams * g * 16);
  l.scores = place(a->acc ? (uint64_t)streams * g * l.score_stride * 4 : 0);
  l.total = at;
  return l;
}

// ---- evict -------------------------------------------------------------------

int64_t evict_limit(const mkv_paged_cache* c, const mkv_paged_evict_args* a) {
  return a->max_len ? a->max_len : (int64_t)c->max_pages * c->page_size;
}

// Bytes of the lists of movers and freed slots.  A budget above the bound evicts
// nothing and needs none.
uint64_t evict_list_bytes(const mkv_paged_cache* c, const mkv_paged_evict_args* a) {
  const int64_t m = std::min<int64_t>(a->budget, evict_limit(c, a));
  return ((uint64_t)c->batch * c->n_kv_heads * 2 * m * 4 + 255) & ~(uint64_t)255;
}

// CTAs of a stream, one cluster: doubled while all clusters run at once (8 CTAs:
// up to 8 streams; 16 clusters of 8 take two turns) and a CTA keeps 8192 slots.
// Us with 1, 2, 4 and 8 CTAs, fp16 rows of 128: 64 streams of 4096 cut to 2048:
// 22.6, 25.3, 35.8, 82.8; 16 of 16384: 22.4, 20.5, 21.1, 38.3; 32 of 32768: 31.1,
// 31.3, 30.2, 59.1; 8 of 131072: 42.0, 35.9, 31.5, 28.7.
int evict_ranks(const mkv_paged_cache* c, int64_t limit, int sms) {
  const int64_t streams = (int64_t)c->batch * c->n_kv_heads;
  int R = 1;
  while (R < 8 && streams * 2 * R <= sms && (R < 4 || streams <= 8) && limit >= 16384 * (int64_t)R) R *= 2;
  return R;
}

uint64_t evict_bytes(const mkv_paged_cache* c, const mkv_paged_evict_args* a, int sms) {
  const int64_t limit = evict_limit(c, a);
  return evict_list_bytes(c, a) +
         (uint64_t)c->batch * c->n_kv_heads * evict_list_slots(limit, evict_ranks(c, limit, sms)) * 8;
}

const char* check_evict(const mkv_paged_cache* c, const mkv_paged_evict_args* a) {
  if (const char* e = check_cache(c)) return e;
  if (!a) return "mkv_paged_evict: NULL arguments";
  if (a->max_len < 0 || a->max_len > (int64_t)c->max_pages * c->page_size)
    return "mkv_paged_evict: max_len must be 0..max_pages * page_size";
  const int64_t limit = evict_limit(c, a);
  if (a->budget < 1) return "mkv_paged_evict: budget must be >= 1";
  if (a->sink < 0 || a->recent < 0 || (int64_t)a->sink + a->recent > a->budget)
    return "mkv_paged_evict: sink and recent must be >= 0 and together at most the budget";
  if (a->meta_stride < limit) return "mkv_paged_evict: meta_stride must be >= max_len";
  if (a->out_stride < std::min<int64_t>(a->budget, limit))
    return "mkv_paged_evict: out_stride must be >= min(budget, max_len)";
  const int64_t streams = (int64_t)c->batch * c->n_kv_heads;
  if (streams * 8 > kMaxGrid || streams * up(std::min<int64_t>(a->budget, limit), 64) > kMaxGrid)
    return "mkv_paged_evict: too many streams";
  return nullptr;
}

}  // namespace

namespace mkv {

cudaError_t encode_rows_map(CUtensorMap* map, const void* base, int64_t rows, int row_bytes, int box_rows) {
  // the driver's encoder, looked up once: it is the process's, not a device's
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(
        e == cudaSuccess && found == cudaDriverEntryPointSuccess ? fn : nullptr);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint32_t w = row_bytes < 128 ? row_bytes : 128;
  // columns of w bytes, rows, column groups of a row
  const cuuint64_t dim[3] = {w, (cuuint64_t)rows, (cuuint64_t)row_bytes / w};
  const cuuint64_t stride[2] = {(cuuint64_t)row_bytes, w};
  const cuuint32_t box[3] = {w, (cuuint32_t)box_rows, (cuuint32_t)row_bytes / w};
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dim, stride, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace mkv

extern "C" {

mkv_status mkv_rope_plan_init(const mkv_rope_config* cfg, mkv_rope_plan* plan) {
  if (!cfg || !plan) return bad("mkv_rope_plan_init: NULL argument");
  const mkv_rope_config& c = *cfg;
  if (c.head_dim < 1 || c.head_dim > 4096) return bad("mkv_rope_plan_init: head_dim must be 1..4096");
  if (c.rot_dim < 2 || c.rot_dim % 2 != 0 || c.rot_dim > c.head_dim || c.rot_dim > 2 * MKV_ROPE_MAX_PAIRS)
    return bad("mkv_rope_plan_init: rot_dim must be even, 2..min(head_dim, 256)");
  if (c.interleaved < 0 || c.interleaved > 1) return bad("mkv_rope_plan_init: interleaved must be 0 or 1");
  if (c.scaling < MKV_ROPE_NONE || c.scaling > MKV_ROPE_BANDED) return bad("mkv_rope_plan_init: unknown scaling");
  if (!(c.base > 1.0) || !std::isfinite(c.base)) return bad("mkv_rope_plan_init: base must be > 1 and finite");
  if (c.scaling != MKV_ROPE_NONE && (!(c.factor >= 1.0) || !std::isfinite(c.factor)))
    return bad("mkv_rope_plan_init: factor must be >= 1 and finite");
  if (c.scaling == MKV_ROPE_NTK && c.rot_dim < 4) return bad("mkv_rope_plan_init: NTK scaling needs rot_dim >= 4");
  if (c.scaling >= MKV_ROPE_YARN && (!(c.original > 0.0) || !std::isfinite(c.original)))
    return bad("mkv_rope_plan_init: original must be > 0 and finite");
  if (c.scaling == MKV_ROPE_YARN &&
      (!(c.beta_slow > 0.0) || !(c.beta_fast >= c.beta_slow) || !std::isfinite(c.beta_fast)))
    return bad("mkv_rope_plan_init: beta_fast >= beta_slow > 0");
  if (c.scaling == MKV_ROPE_BANDED &&
      (!(c.low_freq > 0.0) || !(c.high_freq > c.low_freq) || !std::isfinite(c.high_freq)))
    return bad("mkv_rope_plan_init: 0 < low_freq < high_freq");
  if (!(c.attn_factor >= 0.0) || !std::isfinite((float)c.attn_factor))
    return bad("mkv_rope_plan_init: attn_factor must be >= 0 and finite");

  std::memset(plan, 0, sizeof(*plan));
  plan->head_dim = c.head_dim;
  plan->rot_dim = c.rot_dim;
  plan->interleaved = c.interleaved;
  const double n = c.rot_dim;
  double base = c.base, mult = 1.0;
  if (c.scaling == MKV_ROPE_NTK) base *= std::pow(c.factor, n / (n - 2.0));
  if (c.scaling == MKV_ROPE_YARN) mult = 0.1 * std::log(c.factor) + 1.0;
  if (c.attn_factor > 0.0) mult = c.attn_factor;
  plan->mult = (float)mult;
  // YaRN: index of the pair that turns `turns` times over the original context
  auto pair_of = [&](double turns) {
    return n * std::log(c.original / (turns * kTwoPi)) / (2.0 * std::log(c.base));
  };
  double lo = 0.0, hi = 1.0;
  if (c.scaling == MKV_ROPE_YARN) {
    lo = std::max(0.0, std::floor(pair_of(c.beta_fast)));
    hi = std::min(n - 1.0, std::ceil(pair_of(c.beta_slow)));
  }
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / n);
    if (c.scaling == MKV_ROPE_LINEAR) {
      f /= c.factor;
    } else if (c.scaling == MKV_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      f = f * (1.0 - ramp) + f / c.factor * ramp;
    } else if (c.scaling == MKV_ROPE_BANDED) {
      const double turns = c.original * f / kTwoPi;   // original / wavelength
      const double keep =
          std::min(1.0, std::max(0.0, (turns - c.low_freq) / (c.high_freq - c.low_freq)));
      f = f * keep + f / c.factor * (1.0 - keep);
    }
    // f <= 1 radian, so the fraction of a turn is below 2^62 of 2^64
    plan->turn[i] = (uint64_t)std::llround(std::ldexp(f / kTwoPi, 64));
  }
  return MKV_OK;
}

mkv_status mkv_rope(const mkv_rope_plan* plan, const mkv_rope_args* a, mkv_stream_t stream) {
  if (!plan || !a) return bad("mkv_rope: NULL plan or arguments");
  if (const char* e = check_plan(plan)) return bad(e);
  if (a->batch < 0 || a->heads < 0 || a->tokens < 0) return bad("mkv_rope: negative size");
  if (a->batch > 65535 || a->heads > 65535) return bad("mkv_rope: batch and heads must be <= 65535");
  if (a->dtype != MKV_DT_F16 && a->dtype != MKV_DT_BF16 && a->dtype != MKV_DT_F32)
    return bad("mkv_rope: dtype must be F16, BF16 or F32");
  if (a->transposed < 0 || a->transposed > 1) return bad("mkv_rope: transposed must be 0 or 1");
  if (a->batch == 0 || a->heads == 0 || a->tokens == 0) return MKV_OK;
  if (!a->x || !a->out) return bad("mkv_rope: NULL x or out");
  if (!a->pos && (int64_t)a->first_pos + a->tokens > (int64_t)1 << 31)
    return bad("mkv_rope: positions exceed 32 bits");
  const int64_t extent[3] = {a->batch, a->tokens, a->heads};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] > 1 && a->out_stride[i] <= 0) return bad("mkv_rope: out's strides must be positive");
    if (a->x == a->out && extent[i] > 1 && a->x_stride[i] != a->out_stride[i])
      return bad("mkv_rope: in place, x and out need the same strides");
  }
  const int es = elem_bytes(a->dtype), V = 16 / es;
  const uintptr_t mask = reinterpret_cast<uintptr_t>(a->x) | reinterpret_cast<uintptr_t>(a->out);
  if (mask & (uintptr_t)(es - 1)) return bad("mkv_rope: x and out must be aligned to their elements");
  bool vec = (mask & 15u) == 0 && plan->head_dim % V == 0 &&
             plan->rot_dim % (plan->interleaved ? V : 2 * V) == 0;
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1 && (a->x_stride[i] % V != 0 || a->out_stride[i] % V != 0)) vec = false;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.plan = *plan;
  p.x = a->x;
  p.out = a->out;
  p.pos = a->pos;
  for (int i = 0; i < 3; ++i) p.xs[i] = a->x_stride[i], p.os[i] = a->out_stride[i];
  p.pos_stride = a->pos_stride;
  p.tokens = a->tokens;
  p.batch = a->batch;
  p.heads = a->heads;
  p.first_pos = a->first_pos;
  p.sign = a->transposed ? -1.f : 1.f;
  const int rest = plan->head_dim - plan->rot_dim;
  if (vec) {
    p.rot_units = plan->interleaved ? plan->rot_dim / V : plan->rot_dim / (2 * V);
    p.units = p.rot_units + rest / V;
  } else {
    p.rot_units = plan->rot_dim / 2;
    p.units = p.rot_units + rest;
  }
  if (p.tokens > kMaxGrid / p.units * 256) return bad("mkv_rope: too many tokens");
  int sms = 0;
  mkv_status s = sm_count(&sms);
  if (s != MKV_OK) return s;
  p.heads_per = heads_per_thread((int64_t)a->batch * a->tokens * p.units, a->heads, (int64_t)sms * 2048, 8);
  CKP(launch_rope(p, a->dtype, vec, reinterpret_cast<cudaStream_t>(stream)));
  return MKV_OK;
}

mkv_status mkv_paged_validate(const mkv_paged_cache* cache) {
  const char* e = check_cache(cache);
  return e ? bad(e) : MKV_OK;
}

mkv_status mkv_paged_append(const mkv_paged_cache* c, const mkv_rope_plan* plan,
                            const mkv_paged_append_args* a, mkv_stream_t stream) {
  if (const char* e = check_cache(c)) return bad(e);
  if (!a) return bad("mkv_paged_append: NULL arguments");
  if (plan) {
    if (const char* e = check_plan(plan)) return bad(e);
    if (plan->head_dim != c->head_dim) return bad("mkv_paged_append: the plan's head_dim is not the cache's");
    if (plan->rot_dim % (plan->interleaved ? 8 : 16) != 0)
      return bad("mkv_paged_append: rot_dim must be a multiple of 16 (half pairs) or 8 (interleaved)");
  }
  if (a->n < 0) return bad("mkv_paged_append: n must be >= 0");
  if (!is16(a->in_dtype) || (c->dtype != MKV_DT_E4M3 && a->in_dtype != c->dtype))
    return bad("mkv_paged_append: inputs must be F16 or BF16, of the cache's type unless that is E4M3");
  if (a->n == 0) return MKV_OK;
  if (!a->k || !a->v || !a->slot) return bad("mkv_paged_append: NULL k, v or slot");
  if (!a->seq && a->n > c->batch) return bad("mkv_paged_append: more tokens than sequences need seq");
  if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->q) || !aligned16(a->q_out))
    return bad("mkv_paged_append: k, v, q and q_out must be 16-byte aligned");
  if (a->q && (!a->q_out || a->n_q_heads < 1 || a->n_q_heads > 1 << 20))
    return bad("mkv_paged_append: q needs q_out and n_q_heads >= 1");
  for (int i = 0; i < 2; ++i) {
    const int64_t kv_extent = i == 0 ? a->n : c->n_kv_heads, q_extent = i == 0 ? a->n : a->n_q_heads;
    if (!stride8(a->k_stride[i], kv_extent) || !stride8(a->v_stride[i], kv_extent) ||
        (a->q && (!stride8(a->q_stride[i], q_extent) || !stride8(a->q_out_stride[i], q_extent))))
      return bad("mkv_paged_append: strides must be multiples of 8 elements");
    if (a->q && a->q_out_stride[i] <= 0 && q_extent > 1)
      return bad("mkv_paged_append: q_out's strides must be positive");
    if (a->q && a->q == a->q_out && q_extent > 1 && a->q_stride[i] != a->q_out_stride[i])
      return bad("mkv_paged_append: in place, q and q_out need the same strides");
  }
  if ((a->acc || a->pos_meta) && a->meta_stride < 1) return bad("mkv_paged_append: meta_stride must be >= 1");
  AppendRowsParams p;
  std::memset(&p, 0, sizeof(p));
  if (plan) p.plan = *plan;
  p.c = *c;
  p.a = *a;
  const int rot = p.plan.rot_dim;
  p.rot_units = p.plan.interleaved ? rot / 8 : rot / 16;
  p.units = p.rot_units + (c->head_dim - rot) / 8;
  p.heads_total = 2 * c->n_kv_heads + (a->q ? a->n_q_heads : 0);
  if (a->n > kMaxGrid / p.units * 256) return bad("mkv_paged_append: too many tokens");
  int sms = 0;
  mkv_status s = sm_count(&sms);
  if (s != MKV_OK) return s;
  p.heads_per = heads_per_thread(a->n * p.units, p.heads_total, (int64_t)sms * 2048, 16);
  while (up(p.heads_total, p.heads_per) > 65535) p.heads_per *= 2;
  CKP(launch_append_rows(p, reinterpret_cast<cudaStream_t>(stream)));
  return MKV_OK;
}

uint64_t mkv_paged_decode_workspace(const mkv_paged_cache* c, const mkv_paged_decode_args* a) {
  if (const char* e = check_decode(c, a)) {
    bad(e);
    return 0;
  }
  int sms = 0;
  if (sm_count(&sms) != MKV_OK) return 0;
  return decode_layout(c, a, sms).total;
}

mkv_status mkv_paged_decode(const mkv_paged_cache* c, const mkv_paged_decode_args* a, mkv_stream_t stream) {
  if (const char* e = check_decode(c, a)) return bad(e);
  if (!a->q || !a->out || !a->seq_lens) return bad("mkv_paged_decode: NULL q, out or seq_lens");
  if (!aligned16(a->q) || !aligned16(a->out)) return bad("mkv_paged_decode: q and out must be 16-byte aligned");
  if (!stride8(a->q_stride[0], c->batch) || !stride8(a->q_stride[1], a->n_q_heads))
    return bad("mkv_paged_decode: q's strides must be multiples of 8 elements");
  if (a->acc && a->acc_stride < decode_limit(c, a)) return bad("mkv_paged_decode: acc_stride must be >= max_len");
  if (!a->workspace || !aligned16(a->workspace)) return bad("mkv_paged_decode: workspace must be 16-byte aligned");
  int sms = 0;
  mkv_status s = sm_count(&sms);
  if (s != MKV_OK) return s;
  const DecodeLayout l = decode_layout(c, a, sms);
  if (a->workspace_bytes < l.total) return bad("mkv_paged_decode: workspace too small");
  if (a->acc && (int64_t)c->batch * c->n_kv_heads * up(l.limit, 1024) > kMaxGrid)
    return bad("mkv_paged_decode: too many tokens for accumulated weights");
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.kp = static_cast<const uint8_t*>(c->k_pages);
  p.vp = static_cast<const uint8_t*>(c->v_pages);
  p.table = c->page_table;
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.status = c->status;
  p.table_stride = c->table_stride;
  p.rows = (int64_t)c->n_pages * c->n_kv_heads * c->page_size;
  p.B = c->batch;
  p.H = c->n_kv_heads;
  p.g = a->n_q_heads / c->n_kv_heads;
  p.n_pages = c->n_pages;
  p.bpp = c->page_size / PA_BLOCK;
  p.limit = (int)l.limit;
  p.q = a->q;
  p.q_sb = a->q_stride[0];
  p.q_sh = a->q_stride[1];
  p.q_bf16 = a->q_dtype == MKV_DT_BF16;
  p.out = a->out;
  p.out_type = a->out_dtype;
  p.lse = a->lse;
  p.lens = a->seq_lens;
  const double scale = a->scale > 0.f ? (double)a->scale : 1.0 / std::sqrt((double)c->head_dim);
  p.scale2 = (float)(scale * 1.4426950408889634);
  p.acc = a->acc;
  p.acc_stride = a->acc_stride;
  p.part_o = reinterpret_cast<float*>(ws + l.part_o);
  p.part_ml = reinterpret_cast<float*>(ws + l.part_ml);
  p.stat = reinterpret_cast<float4*>(ws + l.stat);
  p.pre = reinterpret_cast<int64_t*>(ws + l.pre);
  p.scores = a->acc ? reinterpret_cast<float*>(ws + l.scores) : nullptr;
  p.score_stride = l.score_stride;
  p.sms = sms;
  p.G = l.G;
  p.min_blocks = kMinBlocks;
  p.split = l.split;
  p.cluster = l.cluster;
  p.piece_load = kPieceLoad;
  p.tail16 = kTail16;
  p.tail_from = kTailFrom;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (c->head_dim) {
    case 64: CKP(launch_paged_attn_64(p, c->dtype, st)); break;
    case 128: CKP(launch_paged_attn_128(p, c->dtype, st)); break;
    default: CKP(launch_paged_attn_256(p, c->dtype, st)); break;
  }
  if (l.split) CKP(launch_paged_merge(p, c->head_dim, st));
  if (a->acc) CKP(launch_paged_weights(p, st));
  return MKV_OK;
}

uint64_t mkv_paged_evict_workspace(const mkv_paged_cache* c, const mkv_paged_evict_args* a) {
  if (const char* e = check_evict(c, a)) {
    bad(e);
    return 0;
  }
  int sms = 0;
  if (sm_count(&sms) != MKV_OK) return 0;
  return evict_bytes(c, a, sms);
}

mkv_status mkv_paged_evict(const mkv_paged_cache* c, const mkv_paged_evict_args* a, mkv_stream_t stream) {
  if (const char* e = check_evict(c, a)) return bad(e);
  if (!a->acc || !a->pos || !a->acc_out || !a->pos_out || !a->seq_lens || !a->next_pos || !a->lens_out || !a->src)
    return bad("mkv_paged_evict: NULL pointer");
  if ((static_cast<const void*>(a->acc_out) == a->acc || static_cast<const void*>(a->pos_out) == a->pos) &&
      a->out_stride != a->meta_stride)
    return bad("mkv_paged_evict: in place, out_stride must be meta_stride");
  if (!a->workspace || !aligned16(a->workspace)) return bad("mkv_paged_evict: workspace must be 16-byte aligned");
  if (a->workspace_bytes < evict_list_bytes(c, a)) return bad("mkv_paged_evict: workspace too small");
  int sms = 0;
  mkv_status s = sm_count(&sms);
  if (s != MKV_OK) return s;
  if (a->workspace_bytes < evict_bytes(c, a, sms)) return bad("mkv_paged_evict: workspace too small");
  EvictParams p;
  std::memset(&p, 0, sizeof(p));
  p.kp = static_cast<uint8_t*>(c->k_pages);
  p.vp = static_cast<uint8_t*>(c->v_pages);
  p.table = c->page_table;
  p.status = c->status;
  p.table_stride = c->table_stride;
  p.B = c->batch;
  p.H = c->n_kv_heads;
  p.n_pages = c->n_pages;
  p.ps = c->page_size;
  p.row_bytes = c->head_dim * elem_bytes(c->dtype);
  p.limit = (int)evict_limit(c, a);
  p.acc = a->acc;
  p.pos = a->pos;
  p.acc_out = a->acc_out;
  p.pos_out = a->pos_out;
  p.lens = a->seq_lens;
  p.next_pos = a->next_pos;
  p.lens_out = a->lens_out;
  p.src = a->src;
  p.meta_stride = a->meta_stride;
  p.out_stride = a->out_stride;
  p.budget = a->budget;
  p.sink = a->sink;
  p.recent = a->recent;
  const uint64_t lists = evict_list_bytes(c, a);
  p.lists = static_cast<int32_t*>(a->workspace);
  p.R = evict_ranks(c, p.limit, sms);
  p.listed = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a->workspace) + lists);
  p.list_slots = evict_list_slots(p.limit, p.R);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  CKP(launch_evict_select(p, st));
  CKP(launch_evict_move(p, st));
  return MKV_OK;
}

mkv_status mkv_paged_check(int32_t* status) {
  if (!status) return bad("mkv_paged_check: NULL status word");
  CKP(cudaDeviceSynchronize());
  int32_t v = 0;
  CKP(cudaMemcpy(&v, status, sizeof(v), cudaMemcpyDeviceToHost));
  if (v == 0) return MKV_OK;
  CKP(cudaMemset(status, 0, sizeof(v)));
  CKP(cudaDeviceSynchronize());
  // the graver first: outputs are undefined after a wait that gave up, defined otherwise
  if (v & DEV_ERR_TIMEOUT)
    return set_error(MKV_ERR_TIMEOUT, v & DEV_ERR_CHECK ? "a bounded device-side wait gave up; a page, slot, sequence or "
                                                          "length lay outside the paged cache too"
                                                        : "a bounded device-side wait gave up");
  return set_error(MKV_ERR_DEVICE_CHECK, "a page, slot, sequence or length lay outside the paged cache");
}

}  // extern "C"
