// Host side of the calls between projections and caches: norms with rotation,
// attention of prompts and of several new tokens over the paged cache.  No state
// is kept between calls.
#include "api_common.cuh"
#include "attend_internal.cuh"

using namespace mkv;

namespace {

constexpr int kMaxGroup = 128;

// A scale or a cap of scores: 0 (a default), or a number that log2(e) times leaves finite.
bool factor_ok(float x) { return x >= 0.f && x <= 0x1p127f; }

// ---- norms -------------------------------------------------------------------

// Checks the sizes of a norm call and fills the part of its parameters that no
// pointer is needed for; *form as in launch_norm_rope.
const char* norm_sizes(const mkv_rope_plan* plan, const mkv_norm_rope_args* a, bool grad, NormRopeParams* p, int* form) {
  if (!plan || !a) return "mkv_norm_rope: NULL plan or arguments";
  if (const char* e = check_plan(plan)) return e;
  if (plan->head_dim > 256) return "mkv_norm_rope: head_dim must be <= 256";
  if (a->batch < 0 || a->heads[0] < 0 || a->heads[1] < 0 || a->tokens < 0) return "mkv_norm_rope: negative size";
  if (a->batch > 65535 || a->heads[0] > 65535 || a->heads[1] > 65535)
    return "mkv_norm_rope: batch and heads must be <= 65535";
  if (a->tokens > (int64_t)1 << 31) return "mkv_norm_rope: too many tokens";
  if (a->dtype != MKV_DT_F16 && a->dtype != MKV_DT_BF16 && a->dtype != MKV_DT_F32)
    return "mkv_norm_rope: dtype must be F16, BF16 or F32";
  if (a->weight_dtype != a->dtype && a->weight_dtype != MKV_DT_F32)
    return "mkv_norm_rope: weights must be of x's type or F32";
  if (!(a->eps >= 0.f) || std::isinf(a->eps)) return "mkv_norm_rope: eps must be >= 0 and finite";
  if (!std::isfinite(a->weight_offset)) return "mkv_norm_rope: weight_offset must be finite";
  const int es = elem_bytes(a->dtype), bytes = norm_vector_bytes(es == 2, grad), V = bytes / es;
  bool vec = plan->head_dim % V == 0 && plan->rot_dim % (plan->interleaved ? V : 2 * V) == 0;
  const int64_t extent[3] = {a->batch, a->tokens, 0};
  for (int s = 0; s < 2; ++s) {
    if (a->heads[s] == 0) continue;
    uintptr_t mask = reinterpret_cast<uintptr_t>(a->x[s]) | reinterpret_cast<uintptr_t>(a->out[s]);
    if (grad) mask |= reinterpret_cast<uintptr_t>(a->grad[s]);
    if (mask & (uintptr_t)(es - 1)) return "mkv_norm_rope: tensors must be aligned to their elements";
    vec = vec && (mask & (uintptr_t)(bytes - 1)) == 0;
    for (int i = 0; i < 3; ++i) {
      const int64_t n = i < 2 ? extent[i] : a->heads[s];
      if (n <= 1) continue;
      vec = vec && a->x_stride[s][i] % V == 0 && a->out_stride[s][i] % V == 0 && !(grad && a->grad_stride[s][i] % V);
    }
  }
  std::memset(p, 0, sizeof(*p));
  p->plan = *plan;
  const int rest = plan->head_dim - plan->rot_dim;
  *form = !vec ? 0 : plan->interleaved ? 2 : 1;
  p->rot_units = *form == 0 ? plan->rot_dim / 2 : *form == 2 ? plan->rot_dim / V : plan->rot_dim / (2 * V);
  p->units = p->rot_units + (vec ? rest / V : rest);
  p->lanes = 1;
  while (p->lanes < 32 && (p->lanes < p->units || *form == 0)) p->lanes *= 2;
  return nullptr;
}

// Blocks of both sides an SM: those that run at once.  8192 x 4 bf16 tokens of 16 + 16 heads
// of 128: 94.5 us with 2, 112 with 3, 101 with 4 (32 + 8: 128, 149, 128); a gradient's sums
// of a block go through memory (84 us with 2, 94 with 4).
constexpr int kNormBlocks = 2;

// Heads a group of lanes takes, a side's items and blocks.
void norm_grid(const mkv_norm_rope_args* a, int sms, NormRopeParams* p) {
  const int64_t rows = (int64_t)a->batch * a->tokens;
  const int per_block = 256 / p->lanes;
  const int heads[2] = {a->heads[0], a->heads[1]};
  p->heads_per = heads_per_thread(rows * p->lanes, heads[0] + heads[1], (int64_t)sms * 2048, 16);
  int64_t need[2], all = 0;
  for (int s = 0; s < 2; ++s) {
    p->chunks[s] = (int)up(heads[s], p->heads_per);
    p->items[s] = rows * p->chunks[s];
    need[s] = up(p->items[s], per_block);
    all += need[s];
  }
  const int64_t most = (int64_t)sms * kNormBlocks;
  for (int s = 0; s < 2; ++s) {
    const int64_t share = heads[s] * most / (heads[0] + heads[1]);
    p->blocks[s] = (int)(all <= most ? need[s] : std::min(need[s], std::max<int64_t>(share, 1)));
  }
}

// A block more than the share of each side, at most.
uint64_t norm_workspace(const mkv_rope_plan* plan, int sms) {
  return (uint64_t)(sms * kNormBlocks + 2) * plan->head_dim * 4;
}

mkv_status norm_call(const mkv_rope_plan* plan, const mkv_rope_axes* axes, const mkv_norm_rope_args* a, bool grad,
                     mkv_stream_t stream) {
  NormRopeParams p;
  int form = 0;
  if (const char* e = norm_sizes(plan, a, grad, &p, &form)) return bad(e);
  if (axes)
    if (const char* e = check_axes(axes, plan)) return bad(e);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wants = grad && (a->weight_grad[0] || a->weight_grad[1]);
  for (int s = 0; s < 2; ++s) {
    if (grad && a->weight_grad[s] && !a->heads[s] && s == 1 && !a->x[1]) return bad("mkv_norm_rope: a weight_grad without x");
    if (grad && a->weight_grad[s] && !a->weight[s]) return bad("mkv_norm_rope: a weight_grad without a weight");
  }
  if (a->batch == 0 || a->tokens == 0 || a->heads[0] + a->heads[1] == 0) {
    for (int s = 0; s < 2; ++s)
      if (grad && a->weight_grad[s]) CKP(cudaMemsetAsync(a->weight_grad[s], 0, 4 * (size_t)plan->head_dim, st));
    return MKV_OK;
  }
  if (axes && !a->pos) return bad("mkv_norm_rope: axes need pos");
  if (!a->pos && (int64_t)a->first_pos + a->tokens > (int64_t)1 << 31) return bad("mkv_norm_rope: positions exceed 32 bits");
  const int64_t extent[2] = {a->batch, a->tokens};
  for (int s = 0; s < 2; ++s) {
    if (a->heads[s] == 0) continue;
    if (!a->x[s] || !a->out[s] || (grad && !a->grad[s])) return bad("mkv_norm_rope: NULL x, out or grad");
    for (int i = 0; i < 3; ++i) {
      const int64_t n = i < 2 ? extent[i] : a->heads[s];
      if (n <= 1) continue;
      if (a->out_stride[s][i] <= 0) return bad("mkv_norm_rope: out's strides must be positive");
      if ((a->x[s] == a->out[s] && a->x_stride[s][i] != a->out_stride[s][i]) ||
          (grad && a->grad[s] == a->out[s] && a->grad_stride[s][i] != a->out_stride[s][i]))
        return bad("mkv_norm_rope: in place, out needs its input's strides");
      p.xs[s][i] = a->x_stride[s][i];
      p.os[s][i] = a->out_stride[s][i];
      if (grad) p.gs[s][i] = a->grad_stride[s][i];
    }
    const int wb = elem_bytes(a->weight_dtype);
    if (reinterpret_cast<uintptr_t>(a->weight[s]) & (uintptr_t)(wb - 1)) return bad("mkv_norm_rope: weights must be aligned to their elements");
    p.x[s] = a->x[s];
    p.out[s] = a->out[s];
    p.grad[s] = grad ? a->grad[s] : nullptr;
    p.weight[s] = a->weight[s];
    p.weight_f32[s] = a->weight_dtype == MKV_DT_F32;
    p.heads[s] = a->heads[s];
  }
  if (axes) p.axes = *axes;
  p.pos = a->pos;
  p.pos_stride = a->pos_stride;
  p.pos_axis_stride = a->pos_axis_stride;
  p.tokens = a->tokens;
  p.batch = a->batch;
  p.first_pos = a->first_pos;
  p.eps = a->eps;
  p.offset = a->weight_offset;
  int sms = 0;
  if (mkv_status s = sm_count(&sms)) return s;
  norm_grid(a, sms, &p);
  if (wants) {
    if (!a->workspace || !aligned16(a->workspace)) return bad("mkv_norm_rope_grad: workspace must be 16-byte aligned");
    if (a->workspace_bytes < norm_workspace(plan, sms)) return bad("mkv_norm_rope_grad: workspace too small");
    p.part = static_cast<float*>(a->workspace);
    for (int s = 0; s < 2; ++s) p.weight_grad[s] = a->weight_grad[s];
  }
  CKP(launch_norm_rope(p, a->dtype, form, grad, st));
  return MKV_OK;
}

// ---- attention ---------------------------------------------------------------

const char* check_prefill(const mkv_prefill_args* a) {
  if (!a) return "mkv_prefill: NULL arguments";
  if (a->batch < 0 || a->batch > 65535) return "mkv_prefill: batch must be 0..65535";
  if (a->n_kv_heads < 1 || a->n_kv_heads > 65535) return "mkv_prefill: n_kv_heads must be 1..65535";
  if (a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads != 0)
    return "mkv_prefill: n_q_heads must be a multiple of n_kv_heads";
  if (a->n_q_heads / a->n_kv_heads > kMaxGroup) return "mkv_prefill: at most 128 query heads per KV head";
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return "mkv_prefill: head_dim must be 64, 128 or 256";
  if (!is16(a->dtype)) return "mkv_prefill: dtype must be F16 or BF16";
  if (a->q_tokens < 0 || a->kv_tokens < 0 || a->q_tokens > (int64_t)1 << 30 || a->kv_tokens > (int64_t)1 << 30)
    return "mkv_prefill: q_tokens and kv_tokens must be 0..2^30";
  if (a->causal < 0 || a->causal > 1) return "mkv_prefill: causal must be 0 or 1";
  if (a->window < 0) return "mkv_prefill: window must be >= 0";
  if (!factor_ok(a->scale)) return "mkv_prefill: scale must be 0..2^127";
  if (!factor_ok(a->cap)) return "mkv_prefill: cap must be 0..2^127";
  if (a->prefix && !a->causal) return "mkv_prefill: prefix goes with causal";
  if ((int64_t)a->batch * a->n_q_heads > kMaxGrid || (double)a->batch * a->n_q_heads * a->q_tokens > 1.0 * kMaxGrid)
    return "mkv_prefill: too many queries";
  return nullptr;
}

const char* check_attend(const mkv_paged_cache* c, const mkv_paged_attend_args* a) {
  if (const char* e = check_cache(c)) return e;
  if (!a) return "mkv_paged_attend: NULL arguments";
  if (a->n < 0 || a->n > 65535) return "mkv_paged_attend: n must be 0..65535";
  if (a->tree && a->n > 64) return "mkv_paged_attend: a tree has at most 64 new tokens";
  if (a->n_q_heads < 1 || a->n_q_heads % c->n_kv_heads != 0)
    return "mkv_paged_attend: n_q_heads must be a multiple of n_kv_heads";
  if (a->n_q_heads / c->n_kv_heads > kMaxGroup) return "mkv_paged_attend: at most 128 query heads per KV head";
  if (!is16(a->q_dtype) || (c->dtype != MKV_DT_E4M3 && a->q_dtype != c->dtype))
    return "mkv_paged_attend: q must be F16 or BF16, of the cache's type unless that is E4M3";
  if (a->max_len < 0 || a->max_len > (int64_t)c->max_pages * c->page_size)
    return "mkv_paged_attend: max_len must be 0..max_pages * page_size";
  if (a->window < 0) return "mkv_paged_attend: window must be >= 0";
  if (!factor_ok(a->scale)) return "mkv_paged_attend: scale must be 0..2^127";
  if (!factor_ok(a->cap)) return "mkv_paged_attend: cap must be 0..2^127";
  if ((double)c->batch * a->n_q_heads * a->n > 1.0 * kMaxGrid) return "mkv_paged_attend: too many queries";
  return nullptr;
}

// Strides that 16-byte copies of rows can walk: positive multiples of 8 elements.
bool strides_ok(const int64_t* s, int64_t e0, int64_t e1, int64_t e2) {
  const int64_t e[3] = {e0, e1, e2};
  for (int i = 0; i < 3; ++i)
    if (e[i] > 1 && (s[i] <= 0 || s[i] % 8 != 0)) return false;
  return true;
}

// How a call's rows and keys are spread, and where its workspace's parts lie.  Few rows are
// held in copies, see the kernel.
struct AttendLayout {
  int copies;
  int tiles, tile_tokens, groups, splits;
  int fold;                                // as in AttendParams
  uint64_t docs, part_o, part_ml, total;   // byte offsets
};

// What a CTA costs apart from its blocks of keys, in blocks, and what a join costs: a new
// token over 32 streams of 32768 slots takes 87 us with these, 97 with 4 and 3.  Parts of
// outputs that a join reads, in the time of a block (some 0.7 us).
constexpr int kCtaBlocks = 8, kJoinBlocks = 4;
constexpr int64_t kJoinBytes = 4 << 20;

// Row tiles: 128 / g tokens each.  Two to a CTA where there are two (each softmax then
// has its own S buffer and K and V are read half as often), but not with heads of 256
// (tensor memory) or 8-bit pages (their second warpgroup widens).
// `reach`: how far from a query the keys that it sees may lie, both ways together; 0: anywhere.
// `mods`: scores are capped or biased.
AttendLayout attend_layout(int B, int H, int g, int D, int64_t nq, int64_t nk, int64_t reach, bool e4m3, bool docs,
                           bool mods, int sms) {
  AttendLayout l;
  l.copies = nq * g <= 32 ? 4 : nq * g <= 64 && e4m3 ? 2 : 1;
  l.tile_tokens = 128 / l.copies / g;
  const int64_t all = up(std::max<int64_t>(nq, 1), l.tile_tokens);
  l.tiles = all > 1 && D < 256 && !e4m3 ? 2 : 1;
  l.groups = (int)up(all, l.tiles);
  const int NB = attend_block(D, l.tiles, e4m3, l.copies > 1);
  const int64_t items = (int64_t)B * H * l.groups;
  int64_t keys = nk;
  if (reach) keys = std::min<int64_t>(nk, reach + l.tiles * l.tile_tokens + NB);
  const int64_t blocks = up(keys, NB);
  l.splits = 1;
  // the new tokens of a tree, 64 at most, see keys from the first one's on
  const int64_t walk = up(reach ? std::min<int64_t>(nk, keys + 64) : keys, NB);
  // a few rows over many keys: parts of the keys, joined by a second kernel
  const int64_t part_bytes = (int64_t)B * H * g * nq * D * 8;      // written and read
  int64_t best = up(items, sms) * (blocks + kCtaBlocks);
  for (int s = 2; s <= 64 && s <= blocks && items * s <= 16 * (int64_t)sms; ++s) {
    const int64_t cost = up(items * s, sms) * (up(blocks, s) + kCtaBlocks) + kJoinBlocks + s * part_bytes / kJoinBytes;
    if (cost < best) best = cost, l.splits = s;
  }
  uint64_t at = 0;
  auto place = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) & ~(uint64_t)255;
    return here;
  };
  if (mods) l.splits = std::max(l.splits, (int)std::min<int64_t>(64, up(walk, AT_PART / NB)));
  l.fold = !mods && up(walk, l.splits) > AT_FOLD / NB ? AT_FOLD / NB - 1 : INT32_MAX;
  const uint64_t rows = l.splits > 1 || l.fold != INT32_MAX ? (uint64_t)items * l.splits * l.tiles * 128 : 0;
  l.docs = place(docs ? (uint64_t)B * up(nk, NB) * 8 : 0);
  l.part_o = place(rows * D * 4);
  l.part_ml = place(l.splits > 1 ? rows * 8 : 0);
  l.total = at;
  return l;
}

// A window reaches both ways without the causal mask, and a prefix past it.
AttendLayout prefill_layout(const mkv_prefill_args* a, int sms) {
  const int64_t reach = a->prefix ? 0 : a->causal ? a->window : 2 * (int64_t)a->window;
  return attend_layout(a->batch, a->n_kv_heads, a->n_q_heads / a->n_kv_heads, a->head_dim, a->q_tokens, a->kv_tokens, reach,
                       false, a->docs != nullptr, a->cap > 0.f || a->slopes, sms);
}

int64_t attend_limit(const mkv_paged_cache* c, const mkv_paged_attend_args* a) {
  const int64_t cap = (int64_t)c->max_pages * c->page_size;
  return a->max_len ? std::min(a->max_len, cap) : cap;
}

AttendLayout paged_layout(const mkv_paged_cache* c, const mkv_paged_attend_args* a, int sms) {
  return attend_layout(c->batch, c->n_kv_heads, a->n_q_heads / c->n_kv_heads, c->head_dim, a->n, attend_limit(c, a),
                       a->window, c->dtype == MKV_DT_E4M3, false, a->cap > 0.f || a->slopes, sms);
}

// Takes over a layout and launches.
mkv_status attend(AttendParams& p, const AttendLayout& l, void* workspace, mkv_stream_t stream) {
  if ((int64_t)p.B * p.H * l.groups * l.splits > kMaxGrid) return bad("attention: too many queries");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.tiles = l.tiles;
  p.copies = l.copies;
  p.tile_tokens = l.tile_tokens;
  p.groups = l.groups;
  p.splits = l.splits;
  p.fold = l.fold;
  p.doc_range = reinterpret_cast<int2*>(ws + l.docs);
  p.part_o = reinterpret_cast<float4*>(ws + l.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + l.part_ml);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.docs) CKP(launch_attend_docs(p, st));
  if (p.copies == 4) CKP(p.D == 256 ? launch_attend_4_256(p, st) : launch_attend_4(p, st));
  else if (p.copies == 2) CKP(launch_attend_2(p, st));
  else switch (p.D) {
    case 64: CKP(launch_attend_64(p, st)); break;
    case 128: CKP(launch_attend_128(p, st)); break;
    default: CKP(launch_attend_256(p, st)); break;
  }
  if (l.splits > 1) CKP(launch_attend_join(p, st));
  return MKV_OK;
}

float scale_of(float scale, int head_dim) {
  return scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)head_dim));
}

}  // namespace

extern "C" {

mkv_status mkv_norm_rope(const mkv_rope_plan* plan, const mkv_rope_axes* axes, const mkv_norm_rope_args* args,
                         mkv_stream_t stream) {
  return norm_call(plan, axes, args, false, stream);
}

mkv_status mkv_norm_rope_grad(const mkv_rope_plan* plan, const mkv_rope_axes* axes, const mkv_norm_rope_args* args,
                              mkv_stream_t stream) {
  return norm_call(plan, axes, args, true, stream);
}

uint64_t mkv_norm_rope_grad_workspace(const mkv_rope_plan* plan, const mkv_norm_rope_args* a) {
  NormRopeParams p;
  int form = 0, sms = 0;
  if (const char* e = norm_sizes(plan, a, true, &p, &form)) {
    bad(e);
    return 0;
  }
  if (!a->weight_grad[0] && !a->weight_grad[1]) return 0;
  if (sm_count(&sms) != MKV_OK) return 0;
  return norm_workspace(plan, sms);
}

uint64_t mkv_prefill_workspace(const mkv_prefill_args* a) {
  if (const char* e = check_prefill(a)) {
    bad(e);
    return UINT64_MAX;
  }
  int sms = 0;
  if (a->batch == 0 || a->q_tokens == 0) return 0;
  return sm_count(&sms) == MKV_OK ? prefill_layout(a, sms).total : UINT64_MAX;
}

mkv_status mkv_prefill(const mkv_prefill_args* a, mkv_stream_t stream) {
  if (const char* e = check_prefill(a)) return bad(e);
  if (a->batch == 0 || a->q_tokens == 0) return MKV_OK;
  if (!a->q || !a->out || (a->kv_tokens && (!a->k || !a->v))) return bad("mkv_prefill: NULL q, k, v or out");
  if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->out))
    return bad("mkv_prefill: q, k, v and out must be 16-byte aligned");
  if (a->out == a->q || a->out == a->k || a->out == a->v) return bad("mkv_prefill: out must not be an input");
  if (!strides_ok(a->q_stride, a->batch, a->q_tokens, a->n_q_heads) ||
      !strides_ok(a->out_stride, a->batch, a->q_tokens, a->n_q_heads) ||
      !strides_ok(a->k_stride, a->batch, a->kv_tokens, a->n_kv_heads) ||
      !strides_ok(a->v_stride, a->batch, a->kv_tokens, a->n_kv_heads))
    return bad("mkv_prefill: strides must be positive multiples of 8 elements");
  int sms = 0;
  if (mkv_status s = sm_count(&sms)) return s;
  const AttendLayout l = prefill_layout(a, sms);
  if (l.total && (!a->workspace || !aligned16(a->workspace))) return bad("mkv_prefill: workspace must be 16-byte aligned");
  if (a->workspace_bytes < l.total) return bad("mkv_prefill: workspace too small");
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.os[i] = a->out_stride[i];
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
  }
  p.B = a->batch;
  p.Hq = a->n_q_heads;
  p.H = a->n_kv_heads;
  p.g = a->n_q_heads / a->n_kv_heads;
  p.D = a->head_dim;
  p.nq = (int)a->q_tokens;
  p.nk = (int)a->kv_tokens;
  p.bf16 = a->dtype == MKV_DT_BF16;
  p.q_lens = a->q_lens;
  p.kv_lens = a->kv_lens;
  p.prefix = a->prefix;
  p.docs = a->docs;
  p.docs_stride = a->docs_stride;
  p.slopes = a->slopes;
  p.causal = a->causal;
  p.window = a->window;
  p.scale = scale_of(a->scale, a->head_dim);
  p.cap = a->cap;
  p.k = a->k;
  p.v = a->v;
  p.status = a->status;
  return attend(p, l, a->workspace, stream);
}

uint64_t mkv_paged_attend_workspace(const mkv_paged_cache* c, const mkv_paged_attend_args* a) {
  if (const char* e = check_attend(c, a)) {
    bad(e);
    return UINT64_MAX;
  }
  int sms = 0;
  if (a->n == 0) return 0;
  if (paged_attend_streams(c, a)) return paged_attend_streaming_workspace(c, a);
  return sm_count(&sms) == MKV_OK ? paged_layout(c, a, sms).total : UINT64_MAX;
}

mkv_status mkv_paged_attend(const mkv_paged_cache* c, const mkv_paged_attend_args* a, mkv_stream_t stream) {
  if (const char* e = check_attend(c, a)) return bad(e);
  if (a->n == 0) return MKV_OK;
  if (!a->q || !a->out || !a->seq_lens) return bad("mkv_paged_attend: NULL q, out or seq_lens");
  if (!aligned16(a->q) || !aligned16(a->out)) return bad("mkv_paged_attend: q and out must be 16-byte aligned");
  if (a->out == a->q) return bad("mkv_paged_attend: out must not be q");
  if (!strides_ok(a->q_stride, c->batch, a->n, a->n_q_heads))
    return bad("mkv_paged_attend: q's strides must be positive multiples of 8 elements");
  if (paged_attend_streams(c, a)) return paged_attend_streaming(c, a, stream);
  int sms = 0;
  if (mkv_status s = sm_count(&sms)) return s;
  const AttendLayout l = paged_layout(c, a, sms);
  if (l.total && (!a->workspace || !aligned16(a->workspace)))
    return bad("mkv_paged_attend: workspace must be 16-byte aligned");
  if (a->workspace_bytes < l.total) return bad("mkv_paged_attend: workspace too small");
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) p.qs[i] = a->q_stride[i];
  p.os[2] = c->head_dim;
  p.os[1] = p.os[2] * a->n_q_heads;
  p.os[0] = p.os[1] * a->n;
  p.B = c->batch;
  p.Hq = a->n_q_heads;
  p.H = c->n_kv_heads;
  p.g = a->n_q_heads / c->n_kv_heads;
  p.D = c->head_dim;
  p.nq = a->n;
  p.nk = (int)attend_limit(c, a);
  p.bf16 = a->q_dtype == MKV_DT_BF16;
  p.q_lens = a->new_lens;
  p.kv_lens = a->seq_lens;
  p.tree = a->tree;
  p.slopes = a->slopes;
  p.causal = 1;
  p.window = a->window;
  p.scale = scale_of(a->scale, c->head_dim);
  p.cap = a->cap;
  p.k = c->k_pages;
  p.v = c->v_pages;
  p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.cache_type = c->dtype;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.status = c->status;
  return attend(p, l, a->workspace, stream);
}

}  // extern "C"
