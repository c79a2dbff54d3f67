// C-ABI entry points of libgdn: host-side validation, the checkpoint planner
// and kernel dispatch.  No HIP call is made before a call is fully validated.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <vector>

#include "cache_internal.h"
#include "gdn.h"
#include "gdn_internal.h"
#include "ssm_internal.h"

namespace {

bool supported_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }
bool supported_chunk(int32_t c) { return c == 16 || c == 32 || c == 64; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks common to every call that takes a gdn_shape.
gdn_status check_shape(const gdn_shape* s) {
  if (!s) return GDN_ERR_NULL;
  if (s->num_qk_heads < 1 || s->num_v_heads < 1) return GDN_ERR_SHAPE;
  if (s->num_v_heads % s->num_qk_heads != 0) return GDN_ERR_UNSUPPORTED;
  if (!supported_dim(s->head_k_dim) || !supported_dim(s->head_v_dim)) return GDN_ERR_UNSUPPORTED;
  if (!supported_chunk(s->chunk)) return GDN_ERR_UNSUPPORTED;
  if (s->io_dtype != GDN_BF16 && s->io_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (s->flags & ~GDN_QK_L2NORM) return GDN_ERR_UNSUPPORTED;
  if (!std::isfinite(s->scale) || !std::isfinite(s->l2_eps) || s->l2_eps < 0.f) return GDN_ERR_SHAPE;
  if (s->q_tok_stride < 0 || s->k_tok_stride < 0 || s->v_tok_stride < 0) return GDN_ERR_SHAPE;
  return GDN_OK;
}

int64_t elem_bytes(const gdn_shape* s) { return s->io_dtype == GDN_BF16 ? 2 : 4; }

// Resolve a token stride (0 = dense) and check that it fits the row, stays
// below 2^23 elements (the kernels address the rows of a chunk with 32-bit
// offsets) and keeps 16-byte alignment of every row.
gdn_status resolve_stride(const gdn_shape* s, int64_t given, int64_t dense, int64_t* out) {
  const int64_t st = given == 0 ? dense : given;
  if (st < dense || st >= (int64_t(1) << 23)) return GDN_ERR_SHAPE;
  if ((st * elem_bytes(s)) % 16 != 0) return GDN_ERR_SHAPE;
  *out = st;
  return GDN_OK;
}

gdn_status check_seqlens(const int32_t* cu, int32_t n_seqs, int32_t n_tokens) {
  if (n_seqs < 0 || n_tokens < 0) return GDN_ERR_SHAPE;
  if (!cu) return GDN_ERR_NULL;
  if (cu[0] != 0) return GDN_ERR_SEQLENS;
  for (int32_t s = 0; s < n_seqs; ++s)
    if (cu[s + 1] < cu[s]) return GDN_ERR_SEQLENS;
  if (cu[n_seqs] != n_tokens) return GDN_ERR_SEQLENS;
  return GDN_OK;
}

// Checkpoints: strictly increasing, each inside a prompt (cu[s] < p <= cu[s+1]).
// Any position works: the scan also ends a chunk at every checkpoint.
gdn_status check_ckpts(const int32_t* cu, int32_t n_seqs, const int32_t* pos, int32_t n) {
  if (n < 0) return GDN_ERR_SHAPE;
  if (n == 0) return GDN_OK;
  if (!pos) return GDN_ERR_NULL;
  int32_t s = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t p = pos[i];
    if (i > 0 && p <= pos[i - 1]) return GDN_ERR_CKPT;
    while (s < n_seqs && cu[s + 1] < p) ++s;
    // skip empty prompts that end exactly at p-1 ... the owner has cu[s] < p
    while (s < n_seqs && !(cu[s] < p && p <= cu[s + 1])) ++s;
    if (s >= n_seqs) return GDN_ERR_CKPT;
  }
  return GDN_OK;
}

// Every slot in [0, pool_slots) and no slot twice; the check sorts a copy
// of the n slots, so its host memory is O(n) whatever the pool's size.
template <typename T>
gdn_status check_slots(const T* slots, int64_t n, int64_t pool_slots) {
  std::vector<int64_t> v(slots, slots + n);
  std::sort(v.begin(), v.end());
  for (int64_t i = 0; i < n; ++i)
    if (v[i] < 0 || v[i] >= pool_slots || (i > 0 && v[i] == v[i - 1])) return GDN_ERR_CAPACITY;
  return GDN_OK;
}

int log2_of(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

bool supported_page(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }

// Checks of a cache's handle, and the kernels' form of it.  `data` is false
// where only its sizes are used.
gdn_status check_cache(const gdn_cache* c, bool data, gdn::CacheRef* out) {
  if (!c) return GDN_ERR_NULL;
  if (c->num_kv_heads < 1 || c->n_pages < 1) return GDN_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (!supported_page(c->page)) return GDN_ERR_UNSUPPORTED;
  if (c->code_dtype != GDN_E4M3 && c->code_dtype != GDN_I8) return GDN_ERR_UNSUPPORTED;
  if (data) {
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return GDN_ERR_NULL;
    if (!aligned16(c->k) || !aligned16(c->v)) return GDN_ERR_SHAPE;
  }
  *out = gdn::CacheRef{c->num_kv_heads, c->head_dim, log2_of(c->page), c->n_pages, c->code_dtype == GDN_I8,
                       static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale};
  return GDN_OK;
}

// Token stride of bf16 rows [tokens, heads, d]: 0 = dense, else at least that,
// with every row 16-byte aligned.
gdn_status bf16_stride(int64_t given, int64_t dense, int64_t* out) {
  const int64_t st = given == 0 ? dense : given;
  if (st < dense || st % 8 != 0 || st > INT32_MAX) return GDN_ERR_SHAPE;
  *out = st;
  return GDN_OK;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x && y && x < y + b_bytes && y < x + a_bytes;
}

// A buffer of a call.  One that is written may be its input `twin`, in place.
struct Span {
  const void* p;
  int64_t bytes;
  int twin = -1;
};

// Whether something that is written overlaps an input or something else that
// is written (rows of a stride as a whole, from the first to the last).
template <size_t W, size_t R>
bool overlaps(const Span (&to)[W], const Span (&in)[R]) {
  auto meet = [](const Span& a, const Span& b) { return a.bytes > 0 && b.bytes > 0 && overlap(a.p, a.bytes, b.p, b.bytes); };
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = 0; j < R; ++j)
      if (meet(to[i], in[j]) && !(to[i].twin == (int)j && to[i].p == in[j].p)) return true;
    for (size_t j = 0; j < i; ++j)
      if (meet(to[i], to[j])) return true;
  }
  return false;
}

// A launch holds fewer than 2^32 threads along its first axis.
bool fits_grid(int64_t groups, int64_t threads) { return groups * threads <= UINT32_MAX; }

// What both attention calls check alike.
gdn_status check_attn(const gdn_cache* cache, int32_t Hq, float scale, int32_t n_seqs, int32_t max_pages,
                      const int32_t* kv_len, const int32_t* table, const void* q, int64_t q_stride,
                      const void* out, int64_t rows, gdn::AttnArgs* a) {
  gdn_status st = check_cache(cache, true, &a->c);
  if (st != GDN_OK) return st;
  if (Hq < 1 || max_pages < 0 || !std::isfinite(scale)) return GDN_ERR_SHAPE;
  if ((int64_t)max_pages << a->c.page_shift > 1 << 30) return GDN_ERR_SHAPE;   // positions and steps past them in 32 bits
  if (Hq % a->c.Hkv != 0 || Hq / a->c.Hkv > 64) return GDN_ERR_UNSUPPORTED;
  if (rows * Hq > INT32_MAX) return GDN_ERR_SHAPE;
  if (n_seqs > 0 && (!kv_len || (max_pages > 0 && !table))) return GDN_ERR_NULL;
  if (rows > 0 && (!q || !out)) return GDN_ERR_NULL;
  if ((st = bf16_stride(q_stride, (int64_t)Hq * a->c.dim, &a->q_stride)) != GDN_OK) return st;
  if ((q && !aligned16(q)) || (out && !aligned16(out))) return GDN_ERR_SHAPE;
  if (rows > 0) {   // out must not overlap q
    const char* qb = static_cast<const char*>(q);
    const char* ob = static_cast<const char*>(out);
    const char* qe = qb + ((rows - 1) * a->q_stride + (int64_t)Hq * a->c.dim) * 2;
    const char* oe = ob + rows * Hq * a->c.dim * 2;
    if (qb < oe && ob < qe) return GDN_ERR_SHAPE;
  }
  a->Hq = Hq; a->n_seqs = n_seqs; a->n_tokens = (int32_t)rows; a->scale = scale;
  a->kv_len = kv_len; a->table = table; a->max_pages = max_pages;
  a->max_kv = max_pages << a->c.page_shift;
  a->q = static_cast<const uint16_t*>(q); a->out = static_cast<uint16_t*>(const_cast<void*>(out));
  return GDN_OK;
}

// Checks of a state space layer and what it reads; the kernels' form of it.
gdn_status check_ssm(const gdn_ssm_shape* s, gdn::SsmLayer* l) {
  if (!s) return GDN_ERR_NULL;
  if (s->num_heads < 1 || s->num_groups < 1) return GDN_ERR_SHAPE;
  if (s->num_heads % s->num_groups != 0) return GDN_ERR_UNSUPPORTED;
  if (!supported_dim(s->head_dim) || !supported_dim(s->state_dim)) return GDN_ERR_UNSUPPORTED;
  if (s->flags & ~GDN_SSM_SOFTPLUS) return GDN_ERR_UNSUPPORTED;
  if (!(s->dt_min <= s->dt_max)) return GDN_ERR_SHAPE;   // also NaN
  const int64_t dim = (int64_t)s->num_heads * s->head_dim + 2 * (int64_t)s->num_groups * s->state_dim;
  // the kernels' grids take a head, or a group and eight heads, along their second axis
  if (s->num_heads > 65535 || s->num_groups + (s->num_heads + 7) / 8 > 65535 || dim >= (1 << 23)) return GDN_ERR_SHAPE;
  l->H = s->num_heads; l->G = s->num_groups; l->P = s->head_dim; l->N = s->state_dim; l->conv_dim = (int32_t)dim;
  l->softplus = (s->flags & GDN_SSM_SOFTPLUS) != 0;
  l->dt_min = s->dt_min; l->dt_max = s->dt_max;
  return GDN_OK;
}

// The strides of a state space call's rows and its constants.
gdn_status check_ssm_rows(int64_t rows, int64_t x_given, const void* x, int32_t dt_dtype, int64_t dt_given,
                          const void* dt, const float* A, const float* dt_bias, const float* D, const float* conv_w,
                          const float* conv_b, const void* out, gdn::SsmLayer* l, int64_t* xs, int64_t* dts) {
  if (dt_dtype != GDN_BF16 && dt_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (conv_b && !conv_w) return GDN_ERR_NULL;
  gdn_status st = bf16_stride(x_given, l->conv_dim, xs);
  if (st != GDN_OK) return st;
  *dts = dt_given == 0 ? l->H : dt_given;
  if (*dts < l->H || *dts > INT32_MAX || *xs >= (1 << 23)) return GDN_ERR_SHAPE;
  if ((x && !aligned16(x)) || (conv_w && !aligned16(conv_w)) || (conv_b && !aligned16(conv_b)) || (out && !aligned16(out))) return GDN_ERR_SHAPE;
  if (rows > 0 && (!x || !dt || !A || !out)) return GDN_ERR_NULL;
  l->dt_f32 = dt_dtype == GDN_F32;
  l->A = A; l->dt_bias = dt_bias; l->D = D; l->conv_w = conv_w; l->conv_bias = conv_b;
  return GDN_OK;
}

gdn_status finish_launch(hipError_t e, hipStream_t stream) {
  if (e == hipSuccess) e = hipGetLastError();
  if (e != hipSuccess) {
    (void)hipStreamSynchronize(stream);  // leave nothing of this call in flight
    return GDN_ERR_HIP;
  }
  return GDN_OK;
}

}  // namespace

extern "C" {

const char* gdn_status_string(int32_t status) {
  switch (status) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_NULL: return "GDN_ERR_NULL: a required pointer is NULL";
    case GDN_ERR_SHAPE: return "GDN_ERR_SHAPE: bad count, stride, alignment or size";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED: head dims, chunk, dtype, flags or head ratio not supported";
    case GDN_ERR_SEQLENS: return "GDN_ERR_SEQLENS: cu_seqlens must start at 0, not decrease and end at n_tokens";
    case GDN_ERR_CKPT: return "GDN_ERR_CKPT: checkpoints must increase and each lie inside a prompt";
    case GDN_ERR_CAPACITY: return "GDN_ERR_CAPACITY: output list or workspace too short, or slot outside the pool";
    case GDN_ERR_HIP: return "GDN_ERR_HIP: a HIP call or kernel launch failed";
    default: return "unknown gdn_status";
  }
}

gdn_status gdn_plan_checkpoints(const int32_t* cu_host, int32_t n_seqs, const int32_t* p0_host,
                                int32_t block, int32_t tail, int32_t* out_pos, int32_t cap,
                                int32_t* n_out) {
  if (!cu_host || !n_out) return GDN_ERR_NULL;
  if (n_seqs < 0 || block < 1 || tail < 0 || cap < 0) return GDN_ERR_SHAPE;
  if (cap > 0 && !out_pos) return GDN_ERR_NULL;
  if (cu_host[0] != 0) return GDN_ERR_SEQLENS;
  for (int32_t s = 0; s < n_seqs; ++s)
    if (cu_host[s + 1] < cu_host[s]) return GDN_ERR_SEQLENS;
  int64_t count = 0;
  std::vector<int64_t> taken;
  for (int32_t s = 0; s < n_seqs; ++s) {
    const int64_t L = cu_host[s + 1] - cu_host[s];
    const int64_t start = p0_host ? p0_host[s] : 0;
    if (start < 0) return GDN_ERR_SHAPE;
    taken.clear();
    // multiples of the block inside (start, start + L]; one in the last
    // `tail` tokens moves back a block; moved ones that hit the start or an
    // earlier one are dropped.  Candidates ascend, so "earlier one" is the
    // last taken.
    for (int64_t c = block * (start / block + 1); c <= start + L; c += block) {
      int64_t p = c;
      if (start + L - p < tail) p -= block;
      if (p <= start) continue;
      if (!taken.empty() && taken.back() >= p) continue;
      taken.push_back(p);
    }
    for (int64_t p : taken) {
      if (count < cap) out_pos[count] = (int32_t)(cu_host[s] + (p - start));
      ++count;
    }
  }
  *n_out = (int32_t)count;
  return count > cap ? GDN_ERR_CAPACITY : GDN_OK;
}

gdn_status gdn_prefill_packed(const gdn_shape* shape, const int32_t* cu_seqlens,
                              const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t n_tokens,
                              const void* q, const void* k, const void* v, const float* g,
                              const float* beta, const float* init_state,
                              const int32_t* ckpt_positions, const int32_t* ckpt_positions_host,
                              int32_t n_ckpt, void* out, float* final_state, float* ckpt_buf,
                              void* stream) {
  gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens);
  if (st != GDN_OK) return st;
  if (n_seqs > 0 && !cu_seqlens) return GDN_ERR_NULL;
  if (n_tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return GDN_ERR_NULL;
  if (n_ckpt < 0) return GDN_ERR_SHAPE;
  if (n_ckpt > 0 && (!ckpt_positions || !ckpt_positions_host || !ckpt_buf)) return GDN_ERR_NULL;
  st = check_ckpts(cu_seqlens_host, n_seqs, ckpt_positions_host, n_ckpt);
  if (st != GDN_OK) return st;
  const int64_t Hqk = shape->num_qk_heads, Hv = shape->num_v_heads;
  const int64_t dk = shape->head_k_dim, dv = shape->head_v_dim;
  int64_t qs, ks, vs;
  if ((st = resolve_stride(shape, shape->q_tok_stride, Hqk * dk, &qs)) != GDN_OK) return st;
  if ((st = resolve_stride(shape, shape->k_tok_stride, Hqk * dk, &ks)) != GDN_OK) return st;
  if ((st = resolve_stride(shape, shape->v_tok_stride, Hv * dv, &vs)) != GDN_OK) return st;
  const void* ptrs[] = {q, k, v, out, init_state, final_state, ckpt_buf};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  if (n_seqs == 0) return GDN_OK;

  gdn::ScanArgs a{};
  a.cu = cu_seqlens; a.n_seqs = n_seqs; a.n_tokens = n_tokens;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.init = init_state;
  a.ckpt = ckpt_positions; a.n_ckpt = n_ckpt;
  a.out = out; a.final_state = final_state; a.ckpt_buf = ckpt_buf;
  a.q_stride = qs; a.k_stride = ks; a.v_stride = vs;
  a.Hqk = (int32_t)Hqk; a.Hv = (int32_t)Hv; a.dk = (int32_t)dk; a.dv = (int32_t)dv;
  a.chunk = shape->chunk; a.bf16 = shape->io_dtype == GDN_BF16;
  a.l2norm = (shape->flags & GDN_QK_L2NORM) != 0;
  a.scale = shape->scale; a.eps = shape->l2_eps;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_prefill(a, s), s);
}

gdn_status gdn_prefill_conv_packed(const gdn_shape* shape, const int32_t* cu_seqlens,
                                   const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t n_tokens,
                                   const void* x, int64_t x_tok_stride, const float* conv_weight,
                                   const void* conv_state_in, void* conv_state_out, const float* g,
                                   const float* beta, const float* init_state,
                                   const int32_t* ckpt_positions, const int32_t* ckpt_positions_host,
                                   int32_t n_ckpt, void* conv_ckpt, void* out, float* final_state,
                                   float* ckpt_buf, void* stream) {
  gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  // the kernel that fuses the conv: bf16, d_k = d_v = 128, 32-token tiles
  if (shape->io_dtype != GDN_BF16 || shape->head_k_dim != 128 || shape->head_v_dim != 128 ||
      shape->chunk < 32)
    return GDN_ERR_UNSUPPORTED;
  st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens);
  if (st != GDN_OK) return st;
  if (n_seqs > 0 && (!cu_seqlens || !conv_weight)) return GDN_ERR_NULL;
  if (n_tokens > 0 && (!x || !g || !beta || !out)) return GDN_ERR_NULL;
  if (n_ckpt < 0) return GDN_ERR_SHAPE;
  if (n_ckpt > 0 && (!ckpt_positions || !ckpt_positions_host || !ckpt_buf)) return GDN_ERR_NULL;
  st = check_ckpts(cu_seqlens_host, n_seqs, ckpt_positions_host, n_ckpt);
  if (st != GDN_OK) return st;
  const int64_t Hqk = shape->num_qk_heads, Hv = shape->num_v_heads;
  const int64_t conv_dim = 2 * Hqk * 128 + Hv * 128;
  int64_t xs;
  if ((st = resolve_stride(shape, x_tok_stride, conv_dim, &xs)) != GDN_OK) return st;
  const void* ptrs[] = {x, conv_weight, conv_state_in, conv_state_out, conv_ckpt, out,
                        init_state, final_state, ckpt_buf};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  if (n_tokens > 0) {  // out must not overlap x
    const char* xb = static_cast<const char*>(x);
    const char* ob = static_cast<const char*>(out);
    const char* xe = xb + ((int64_t)(n_tokens - 1) * xs + conv_dim) * 2;
    const char* oe = ob + (int64_t)n_tokens * Hv * 128 * 2;
    if (xb < oe && ob < xe) return GDN_ERR_SHAPE;
  }
  if (n_seqs == 0) return GDN_OK;

  gdn::ScanArgs a{};
  a.cu = cu_seqlens; a.n_seqs = n_seqs; a.n_tokens = n_tokens;
  a.g = g; a.beta = beta; a.init = init_state;
  a.ckpt = ckpt_positions; a.n_ckpt = n_ckpt;
  a.out = out; a.final_state = final_state; a.ckpt_buf = ckpt_buf;
  a.Hqk = (int32_t)Hqk; a.Hv = (int32_t)Hv; a.dk = 128; a.dv = 128;
  a.chunk = shape->chunk; a.bf16 = 1;
  a.l2norm = (shape->flags & GDN_QK_L2NORM) != 0;
  a.scale = shape->scale; a.eps = shape->l2_eps;
  a.conv_x = x; a.conv_x_stride = xs; a.conv_w = conv_weight;
  a.conv_state_in = conv_state_in; a.conv_state_out = conv_state_out; a.conv_ckpt = conv_ckpt;
  a.conv_dim = (int32_t)conv_dim;
  // conv states written in place: every workgroup of a prompt reads its
  // history first, so the new windows come from a launch of their own after
  const bool in_place = conv_state_out && conv_state_out == conv_state_in;
  a.conv_state_own = conv_state_out && !in_place;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = gdn::launch_prefill(a, s);
  if (e == hipSuccess && in_place) {
    gdn::ConvArgs c{};
    c.cu = cu_seqlens; c.n_seqs = n_seqs; c.n_tokens = n_tokens; c.conv_dim = (int32_t)conv_dim;
    c.x = x; c.x_stride = xs; c.state_in = conv_state_in; c.state_out = conv_state_out; c.bf16 = 1;
    e = gdn::launch_conv_states(c, s);
  }
  return finish_launch(e, s);
}

gdn_status gdn_decode_step(const gdn_shape* shape, int32_t batch, const void* q, const void* k,
                           const void* v, const float* g, const float* beta, float* state,
                           int64_t pool_slots, const int32_t* slot, const int32_t* slot_host,
                           void* out, const float* conv_w, void* conv_state, void* stream) {
  return gdn_decode_tokens(shape, batch, 1, q, k, v, g, beta, state, pool_slots, slot, slot_host, out,
                           nullptr, conv_w, conv_state, stream);
}

gdn_status gdn_decode_tokens(const gdn_shape* shape, int32_t batch, int32_t n_tok, const void* q,
                             const void* k, const void* v, const float* g, const float* beta,
                             float* state, int64_t pool_slots, const int32_t* slot,
                             const int32_t* slot_host, void* out, float* snapshots,
                             const float* conv_w, void* conv_state, void* stream) {
  gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  if (batch < 0 || pool_slots < 0 || n_tok < 1) return GDN_ERR_SHAPE;
  if ((int64_t)batch * n_tok > INT32_MAX) return GDN_ERR_SHAPE;
  if (!conv_w != !conv_state) return GDN_ERR_NULL;   // the conv needs both
  if (batch == 0) return GDN_OK;
  if (!q || !k || !v || !g || !beta || !state || !out) return GDN_ERR_NULL;
  if (slot) {
    if (!slot_host) return GDN_ERR_NULL;
    if ((st = check_slots(slot_host, batch, pool_slots)) != GDN_OK) return st;
  } else if (batch > pool_slots) {
    return GDN_ERR_CAPACITY;
  }
  const int64_t Hqk = shape->num_qk_heads, Hv = shape->num_v_heads;
  const int64_t dk = shape->head_k_dim, dv = shape->head_v_dim;
  int64_t qs, ks, vs;
  if ((st = resolve_stride(shape, shape->q_tok_stride, Hqk * dk, &qs)) != GDN_OK) return st;
  if ((st = resolve_stride(shape, shape->k_tok_stride, Hqk * dk, &ks)) != GDN_OK) return st;
  if ((st = resolve_stride(shape, shape->v_tok_stride, Hv * dv, &vs)) != GDN_OK) return st;
  const void* ptrs[] = {q, k, v, out, state, snapshots, conv_w, conv_state};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  const int64_t conv_dim = 2 * Hqk * dk + Hv * dv;
  if (conv_w && conv_dim > INT32_MAX / 4) return GDN_ERR_SHAPE;

  gdn::DecodeArgs a{};
  a.batch = batch; a.n_tok = n_tok; a.snap = snapshots;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.state = state; a.slot = slot; a.out = out;
  a.conv_w = conv_w; a.conv_state = conv_state; a.conv_dim = (int32_t)conv_dim;
  a.q_stride = qs; a.k_stride = ks; a.v_stride = vs;
  a.Hqk = (int32_t)Hqk; a.Hv = (int32_t)Hv; a.dk = (int32_t)dk; a.dv = (int32_t)dv;
  a.bf16 = shape->io_dtype == GDN_BF16;
  a.l2norm = (shape->flags & GDN_QK_L2NORM) != 0;
  a.scale = shape->scale; a.eps = shape->l2_eps;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_decode(a, s), s);
}

gdn_status gdn_conv1d_silu_packed(const gdn_shape* shape, const int32_t* cu_seqlens,
                                  const int32_t* cu_seqlens_host, int32_t n_seqs,
                                  int32_t n_tokens, const void* x, int64_t x_tok_stride,
                                  const float* weight, const void* conv_state_in, void* y,
                                  int64_t y_tok_stride, void* conv_state_out,
                                  const int32_t* ckpt_positions,
                                  const int32_t* ckpt_positions_host, int32_t n_ckpt,
                                  void* conv_ckpt, void* stream) {
  gdn_status st = check_shape(shape);
  if (st != GDN_OK) return st;
  st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens);
  if (st != GDN_OK) return st;
  if (n_seqs > 0 && !cu_seqlens) return GDN_ERR_NULL;
  if (!weight && n_seqs > 0) return GDN_ERR_NULL;
  if (n_tokens > 0 && (!x || !y)) return GDN_ERR_NULL;
  if (n_ckpt < 0) return GDN_ERR_SHAPE;
  if (n_ckpt > 0 && conv_ckpt && (!ckpt_positions || !ckpt_positions_host)) return GDN_ERR_NULL;
  st = check_ckpts(cu_seqlens_host, n_seqs, ckpt_positions_host, conv_ckpt ? n_ckpt : 0);
  if (st != GDN_OK) return st;
  const int64_t conv_dim = 2LL * shape->num_qk_heads * shape->head_k_dim +
                           (int64_t)shape->num_v_heads * shape->head_v_dim;
  if (conv_dim > INT32_MAX) return GDN_ERR_SHAPE;
  int64_t xs, ys;
  if ((st = resolve_stride(shape, x_tok_stride, conv_dim, &xs)) != GDN_OK) return st;
  if ((st = resolve_stride(shape, y_tok_stride, conv_dim, &ys)) != GDN_OK) return st;
  const void* ptrs[] = {x, y, conv_state_in, conv_state_out, conv_ckpt};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  if (n_tokens > 0) {  // y must not overlap x
    const char* xb = static_cast<const char*>(x);
    const char* yb = static_cast<const char*>(y);
    const int64_t eb = elem_bytes(shape);
    const char* xe = xb + ((int64_t)(n_tokens - 1) * xs + conv_dim) * eb;
    const char* ye = yb + ((int64_t)(n_tokens - 1) * ys + conv_dim) * eb;
    if (xb < ye && yb < xe) return GDN_ERR_SHAPE;
  }
  if (n_seqs == 0) return GDN_OK;

  gdn::ConvArgs a{};
  a.cu = cu_seqlens; a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.conv_dim = (int32_t)conv_dim;
  a.x = x; a.x_stride = xs; a.w = weight; a.state_in = conv_state_in;
  a.y = y; a.y_stride = ys; a.state_out = conv_state_out;
  a.ckpt = conv_ckpt ? ckpt_positions : nullptr; a.n_ckpt = conv_ckpt ? n_ckpt : 0;
  a.conv_ckpt = conv_ckpt; a.bf16 = shape->io_dtype == GDN_BF16;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_conv(a, s), s);
}

gdn_status gdn_snapshot_copy(const void* ckpt_buf, int32_t n, int64_t bytes_each, void* dst_pool,
                             int64_t pool_slots, const int64_t* dst_slot,
                             const int64_t* dst_slot_host, void* wait_event, void* copy_stream,
                             void* done_event) {
  if (n < 0 || pool_slots < 0) return GDN_ERR_SHAPE;
  if (n > 0) {
    if (!ckpt_buf || !dst_pool || !dst_slot || !dst_slot_host) return GDN_ERR_NULL;
    if (bytes_each <= 0 || bytes_each % 16 != 0) return GDN_ERR_SHAPE;
    if (!aligned16(ckpt_buf) || !aligned16(dst_pool)) return GDN_ERR_SHAPE;
    const gdn_status sc = check_slots(dst_slot_host, n, pool_slots);
    if (sc != GDN_OK) return sc;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(copy_stream);
  hipError_t e = hipSuccess;
  if (wait_event) e = hipStreamWaitEvent(s, reinterpret_cast<hipEvent_t>(wait_event), 0);
  if (e != hipSuccess) return GDN_ERR_HIP;
  if (n > 0) {
    // A pool in host memory is bounded by the host link: the gather then runs
    // on one workgroup per item, which keeps the link saturated (faster here
    // than one DMA transfer per item) while holding few CUs.
    hipPointerAttribute_t attr{};
    const hipError_t pe = hipPointerGetAttributes(&attr, dst_pool);
    if (pe != hipSuccess) (void)hipGetLastError();   // not a HIP allocation: treat as device
    const int32_t host_dst = pe == hipSuccess && attr.type == hipMemoryTypeHost;
    gdn::CopyArgs a{ckpt_buf, n, bytes_each, dst_pool, dst_slot, host_dst};
    const gdn_status r = finish_launch(gdn::launch_snapshot_copy(a, s), s);
    if (r != GDN_OK) return r;
  }
  if (done_event) {
    e = hipEventRecord(reinterpret_cast<hipEvent_t>(done_event), s);
    if (e != hipSuccess) return finish_launch(e, s);
  }
  return GDN_OK;
}

gdn_status gdn_plan_pages(int32_t page, int32_t n_seqs, const int32_t* want_len, const int32_t* kv_len,
                          int32_t* kv_len_out, int32_t* block_table, int32_t max_pages,
                          int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                          int32_t n_pages, int32_t* cu_seqlens, int64_t* slot_map, int32_t slot_cap,
                          int32_t* positions, int32_t* status, void* stream) {
  if (!supported_page(page)) return GDN_ERR_UNSUPPORTED;
  if (n_seqs < 0 || max_pages < 0 || n_pages < 1 || slot_cap < 0) return GDN_ERR_SHAPE;
  if (!free_pages || !free_count || !free_count_out || !cu_seqlens) return GDN_ERR_NULL;
  if (n_seqs > 0 && (!want_len || !kv_len || !kv_len_out || !status || (max_pages > 0 && !block_table)))
    return GDN_ERR_NULL;
  if (slot_cap > 0 && !slot_map) return GDN_ERR_NULL;
  gdn::PlanArgs a{};
  a.page_shift = log2_of(page); a.n_seqs = n_seqs; a.max_pages = max_pages; a.n_pages = n_pages;
  a.slot_cap = slot_cap; a.want = want_len; a.kv = kv_len; a.kv_out = kv_len_out; a.table = block_table;
  a.free_pages = free_pages; a.free_count = free_count; a.free_count_out = free_count_out;
  a.cu = cu_seqlens; a.slot = slot_map; a.pos = positions; a.status = status;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_plan_pages(a, s), s);
}

gdn_status gdn_rope_append(const gdn_rope* rope, const gdn_cache* cache, int32_t num_q_heads,
                           const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t n_seqs,
                           int32_t n_tokens, const void* q, int64_t q_tok_stride, const void* k,
                           int64_t k_tok_stride, const void* v, int64_t v_tok_stride,
                           const int32_t* positions, int64_t pos_axis_stride, const int64_t* slot_map,
                           void* q_out, int64_t q_out_tok_stride, void* stream) {
  gdn::AppendArgs a{};
  if (!rope) return GDN_ERR_NULL;
  gdn_status st = check_cache(cache, true, &a.c);
  if (st != GDN_OK) return st;
  if (rope->rot_dim < 0 || rope->rot_dim % 16 != 0 || rope->rot_dim > a.c.dim) return GDN_ERR_UNSUPPORTED;
  if (rope->n_axes < 1 || rope->n_axes > 4 || (rope->adjacent != 0 && rope->adjacent != 1)) return GDN_ERR_UNSUPPORTED;
  if (!std::isfinite(rope->scale) || pos_axis_stride < 0) return GDN_ERR_SHAPE;
  for (int32_t i = 0; i < rope->rot_dim / 2; ++i)
    if (!(std::fabs(rope->freq[i]) <= 65536.f) || rope->axis[i] >= rope->n_axes) return GDN_ERR_SHAPE;
  st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens);
  if (st != GDN_OK) return st;
  if (!q != !q_out) return GDN_ERR_NULL;
  if (q && num_q_heads < 1) return GDN_ERR_SHAPE;
  if (n_seqs > 0 && !cu_seqlens) return GDN_ERR_NULL;
  if (n_tokens > 0 && (!k || !v || !slot_map || (rope->rot_dim > 0 && !positions))) return GDN_ERR_NULL;
  const int64_t d = a.c.dim, hkv = a.c.Hkv, hq = q ? num_q_heads : 1;
  if ((st = bf16_stride(q_tok_stride, hq * d, &a.q_stride)) != GDN_OK) return st;
  if ((st = bf16_stride(q_out_tok_stride, hq * d, &a.qo_stride)) != GDN_OK) return st;
  if ((st = bf16_stride(k_tok_stride, hkv * d, &a.k_stride)) != GDN_OK) return st;
  if ((st = bf16_stride(v_tok_stride, hkv * d, &a.v_stride)) != GDN_OK) return st;
  if (q == q_out && a.q_stride != a.qo_stride) return GDN_ERR_SHAPE;
  const void* ptrs[] = {q, k, v, q_out};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  // a workgroup of 256 per page and head, and per few rows of queries
  if (!fits_grid(((int64_t)n_tokens / cache->page + 2 * (int64_t)n_seqs) * hkv + n_tokens, 256)) return GDN_ERR_SHAPE;
  if (n_tokens == 0) return GDN_OK;
  a.rope.rot = rope->rot_dim; a.rope.n_axes = rope->n_axes; a.rope.adjacent = rope->adjacent;
  a.rope.scale = rope->scale;
  std::copy(rope->freq, rope->freq + 128, a.rope.freq);
  std::copy(rope->axis, rope->axis + 128, a.rope.axis);
  a.Hq = num_q_heads; a.n_seqs = n_seqs; a.n_tokens = n_tokens; a.cu = cu_seqlens;
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v); a.q_out = static_cast<uint16_t*>(q_out);
  a.pos = positions; a.pos_stride = pos_axis_stride; a.slot = slot_map;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_rope_append(a, s), s);
}

gdn_status gdn_cache_gather(const gdn_cache* cache, int32_t n_tokens, const int64_t* slot_map, void* k_out,
                            void* v_out, void* stream) {
  gdn::GatherArgs a{};
  gdn_status st = check_cache(cache, true, &a.c);
  if (st != GDN_OK) return st;
  if (n_tokens < 0 || a.c.Hkv > 65535 || !fits_grid((int64_t)n_tokens / 16 + 1, 256)) return GDN_ERR_SHAPE;
  if (!k_out && !v_out) return GDN_ERR_NULL;
  if (n_tokens > 0 && !slot_map) return GDN_ERR_NULL;
  if ((k_out && !aligned16(k_out)) || (v_out && !aligned16(v_out))) return GDN_ERR_SHAPE;
  if (n_tokens == 0) return GDN_OK;
  a.n_tokens = n_tokens; a.slot = slot_map;
  a.k_out = static_cast<uint16_t*>(k_out); a.v_out = static_cast<uint16_t*>(v_out);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_cache_gather(a, s), s);
}

gdn_status gdn_attn_packed(const gdn_cache* cache, int32_t num_q_heads, float scale, const int32_t* cu_seqlens,
                           const int32_t* cu_seqlens_host, int32_t n_seqs, int32_t n_tokens,
                           const int32_t* kv_len, const int32_t* block_table, int32_t max_pages,
                           const void* q, int64_t q_tok_stride, void* out, void* stream) {
  gdn::AttnArgs a{};
  gdn_status st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens);
  if (st != GDN_OK) return st;
  st = check_attn(cache, num_q_heads, scale, n_seqs, max_pages, kv_len, block_table, q, q_tok_stride, out,
                  n_tokens, &a);
  if (st != GDN_OK) return st;
  if (n_seqs > 0 && !cu_seqlens) return GDN_ERR_NULL;
  // a workgroup of 512 per 256 rows of a prompt and kv head
  if (!fits_grid(((int64_t)n_tokens * (num_q_heads / a.c.Hkv) / 256 + n_seqs) * a.c.Hkv, 512)) return GDN_ERR_SHAPE;
  if (n_tokens == 0) return GDN_OK;
  for (int32_t i = 0; i < n_seqs; ++i) {
    const int32_t n = cu_seqlens_host[i + 1] - cu_seqlens_host[i];
    if (n > gdn::few_rows(a.c.dim) / (num_q_heads / a.c.Hkv)) ++a.many;
    else a.few = std::max(a.few, n);
  }
  // one of 256 per few 16-row tiles of the longest prompt of few rows and kv head
  const int64_t few = (int64_t)a.few * (num_q_heads / a.c.Hkv), tile = 16 * gdn::few_tiles(a.c.dim, (int)few);
  if (!fits_grid((few + tile - 1) / tile * a.c.Hkv, 256)) return GDN_ERR_SHAPE;
  a.cu = cu_seqlens;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_attn_packed(a, s), s);
}

gdn_status gdn_attn_decode_workspace(const gdn_cache* cache, int32_t num_q_heads, int32_t batch, int32_t n_tok,
                                     int32_t max_kv_len, int64_t* bytes) {
  gdn::CacheRef c;
  if (!bytes) return GDN_ERR_NULL;
  const gdn_status st = check_cache(cache, false, &c);
  if (st != GDN_OK) return st;
  if (num_q_heads < 1 || batch < 0 || n_tok < 1 || max_kv_len < 0) return GDN_ERR_SHAPE;
  if ((int64_t)batch * n_tok * num_q_heads > INT32_MAX) return GDN_ERR_SHAPE;
  *bytes = gdn::attn_decode_bytes(c.dim, num_q_heads, batch, n_tok, max_kv_len);
  return GDN_OK;
}

gdn_status gdn_attn_decode(const gdn_cache* cache, int32_t num_q_heads, float scale, int32_t batch,
                           int32_t n_tok, const int32_t* kv_len, const int32_t* block_table,
                           int32_t max_pages, int32_t max_kv_len, const void* q, int64_t q_tok_stride,
                           void* out, void* workspace, int64_t workspace_bytes, void* stream) {
  gdn::AttnArgs a{};
  if (batch < 0 || n_tok < 1 || max_kv_len < 0) return GDN_ERR_SHAPE;
  gdn_status st = check_attn(cache, num_q_heads, scale, batch, max_pages, kv_len, block_table, q, q_tok_stride,
                             out, (int64_t)batch * n_tok, &a);
  if (st != GDN_OK) return st;
  if (max_kv_len > a.max_kv) return GDN_ERR_SHAPE;
  a.max_kv = max_kv_len; a.n_tok = n_tok;
  int64_t need;
  if ((st = gdn_attn_decode_workspace(cache, num_q_heads, batch, n_tok, max_kv_len, &need)) != GDN_OK) return st;
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (workspace_bytes < need) return GDN_ERR_CAPACITY;
  if (workspace && !aligned16(workspace)) return GDN_ERR_SHAPE;
  if (need > 0) {   // nor may the workspace overlap out or q
    const char* wb = static_cast<const char*>(workspace);
    const char* ob = static_cast<const char*>(out);
    const char* qb = static_cast<const char*>(q);
    const int64_t rows = (int64_t)batch * n_tok, row = (int64_t)num_q_heads * a.c.dim * 2;
    if (wb < ob + rows * row && ob < wb + need) return GDN_ERR_SHAPE;
    if (wb < qb + (rows - 1) * a.q_stride * 2 + row && qb < wb + need) return GDN_ERR_SHAPE;
  }
  if (batch == 0) return GDN_OK;
  if (gdn::attn_decode_splits(a.c.dim, max_kv_len) > 65535) return GDN_ERR_SHAPE;
  if (!fits_grid((int64_t)batch * n_tok * num_q_heads, 64)) return GDN_ERR_SHAPE;
  if (batch > 65535 || a.c.Hkv * (((int64_t)n_tok * (num_q_heads / a.c.Hkv) + 15) / 16) > 65535) return GDN_ERR_SHAPE;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_attn_decode(a, workspace, s), s);
}

gdn_status gdn_ssm_prefill_workspace(const gdn_ssm_shape* shape, const int32_t* cu_seqlens_host, int32_t n_seqs,
                                     int32_t n_tokens, int64_t* bytes) {
  gdn::SsmLayer l{};
  if (!bytes) return GDN_ERR_NULL;
  gdn_status st = check_ssm(shape, &l);
  if (st != GDN_OK) return st;
  if ((st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens)) != GDN_OK) return st;
  *bytes = gdn::ssm_scan_bytes(l, n_seqs, cu_seqlens_host);
  return GDN_OK;
}

gdn_status gdn_ssm_prefill_packed(
    const gdn_ssm_shape* shape, const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int32_t n_seqs,
    int32_t n_tokens, const void* x, int64_t x_tok_stride, const float* conv_weight, const float* conv_bias,
    const void* conv_state_in, void* conv_state_out, int32_t dt_dtype, const void* dt, int64_t dt_tok_stride,
    const float* A, const float* dt_bias, const float* D, const float* init_state, const int32_t* ckpt_positions,
    const int32_t* ckpt_positions_host, int32_t n_ckpt, void* conv_ckpt, void* out, float* final_state,
    float* ckpt_buf, void* workspace, int64_t workspace_bytes, void* stream) {
  gdn::SsmScanArgs a{};
  gdn_status st = check_ssm(shape, &a.l);
  if (st != GDN_OK) return st;
  if ((st = check_seqlens(cu_seqlens_host, n_seqs, n_tokens)) != GDN_OK) return st;
  if (n_seqs > 0 && !cu_seqlens) return GDN_ERR_NULL;
  if (n_ckpt < 0) return GDN_ERR_SHAPE;
  if (n_ckpt > 0 && (!ckpt_positions || !ckpt_positions_host || !ckpt_buf)) return GDN_ERR_NULL;
  if ((st = check_ckpts(cu_seqlens_host, n_seqs, ckpt_positions_host, n_ckpt)) != GDN_OK) return st;
  if (!conv_weight && (conv_state_in || conv_state_out || conv_ckpt)) return GDN_ERR_NULL;
  st = check_ssm_rows(n_tokens, x_tok_stride, x, dt_dtype, dt_tok_stride, dt, A, dt_bias, D, conv_weight, conv_bias,
                      out, &a.l, &a.x_stride, &a.dt_stride);
  if (st != GDN_OK) return st;
  const void* ptrs[] = {conv_state_in, conv_state_out, conv_ckpt, init_state, final_state, ckpt_buf, workspace};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  if (!fits_grid(gdn::ssm_scan_groups(a.l, n_seqs, n_tokens), 256) || !fits_grid((int64_t)n_ckpt + n_seqs, 256)) return GDN_ERR_SHAPE;
  const int64_t need = gdn::ssm_scan_bytes(a.l, n_seqs, cu_seqlens_host);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (workspace_bytes < need) return GDN_ERR_CAPACITY;
  const int64_t T = n_tokens, n = n_seqs, H = a.l.H, dim = a.l.conv_dim, head = H * a.l.P * a.l.N * 4;
  const Span in[] = {{x, T > 0 ? ((T - 1) * a.x_stride + dim) * 2 : 0}, {dt, T > 0 ? ((T - 1) * a.dt_stride + H) * (a.l.dt_f32 ? 4 : 2) : 0},
                     {init_state, n * head}, {conv_state_in, n * 6 * dim}, {A, H * 4}, {dt_bias, H * 4}, {D, H * 4},
                     {conv_weight, dim * 16}, {conv_bias, dim * 4}, {cu_seqlens, (n + 1) * 4}, {ckpt_positions, (int64_t)n_ckpt * 4}};
  const Span to[] = {{out, T * H * a.l.P * 2}, {final_state, n * head, 2}, {ckpt_buf, n_ckpt * head}, {conv_state_out, n * 6 * dim, 3},
                     {conv_ckpt, (int64_t)n_ckpt * 6 * dim}, {workspace, need}};
  if (overlaps(to, in)) return GDN_ERR_SHAPE;
  if (n_seqs == 0) return GDN_OK;
  a.cu = cu_seqlens; a.n_seqs = n_seqs; a.n_tokens = n_tokens;
  a.x = static_cast<const uint16_t*>(x); a.dt = dt;
  a.init = init_state; a.final_state = final_state;
  a.ckpt = ckpt_positions; a.n_ckpt = n_ckpt; a.ckpt_buf = ckpt_buf;
  a.out = static_cast<uint16_t*>(out);
  a.conv_in = static_cast<const uint16_t*>(conv_state_in);
  a.conv_out = static_cast<uint16_t*>(conv_state_out);
  a.conv_ckpt = static_cast<uint16_t*>(conv_ckpt);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_ssm_scan(a, cu_seqlens_host, ckpt_positions_host, workspace, s), s);
}

gdn_status gdn_ssm_decode(const gdn_ssm_shape* shape, int32_t batch, int32_t n_tok, const void* x,
                          int64_t x_tok_stride, const float* conv_weight, const float* conv_bias, void* conv_state,
                          int32_t dt_dtype, const void* dt, int64_t dt_tok_stride, const float* A,
                          const float* dt_bias, const float* D, float* state, int64_t pool_slots,
                          const int32_t* slot, const int32_t* slot_host, void* out, float* snapshots, void* stream) {
  gdn::SsmDecodeArgs a{};
  gdn_status st = check_ssm(shape, &a.l);
  if (st != GDN_OK) return st;
  if (batch < 0 || pool_slots < 0 || n_tok < 1) return GDN_ERR_SHAPE;
  if ((int64_t)batch * n_tok > INT32_MAX || !fits_grid(batch, 256)) return GDN_ERR_SHAPE;
  if (!conv_weight != !conv_state) return GDN_ERR_NULL;   // the conv needs both
  st = check_ssm_rows((int64_t)batch * n_tok, x_tok_stride, x, dt_dtype, dt_tok_stride, dt, A, dt_bias, D, conv_weight,
                      conv_bias, out, &a.l, &a.x_stride, &a.dt_stride);
  if (st != GDN_OK) return st;
  const void* ptrs[] = {state, snapshots, conv_state};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return GDN_ERR_SHAPE;
  if (batch == 0) return GDN_OK;
  if (!state) return GDN_ERR_NULL;
  if (slot) {
    if (!slot_host) return GDN_ERR_NULL;
    if ((st = check_slots(slot_host, batch, pool_slots)) != GDN_OK) return st;
  } else if (batch > pool_slots) {
    return GDN_ERR_CAPACITY;
  }
  const int64_t T = (int64_t)batch * n_tok, H = a.l.H, dim = a.l.conv_dim, head = H * a.l.P * a.l.N * 4;
  const Span in[] = {{x, ((T - 1) * a.x_stride + dim) * 2}, {dt, ((T - 1) * a.dt_stride + H) * (a.l.dt_f32 ? 4 : 2)},
                     {A, H * 4}, {dt_bias, H * 4}, {D, H * 4}, {conv_weight, dim * 16}, {conv_bias, dim * 4}, {slot, (int64_t)batch * 4}};
  Span to[] = {{out, T * H * a.l.P * 2}, {snapshots, T * head}, {state, pool_slots * head}, {conv_state, pool_slots * 6 * dim}};
  if (overlaps(to, in)) {
    // the pools as a whole meet something: may be in slots that the call leaves alone
    if (overlap(state, pool_slots * head, conv_state, pool_slots * 6 * dim)) return GDN_ERR_SHAPE;
    for (int32_t b = 0; b < batch; ++b) {
      const int64_t r = slot ? slot_host[b] : b;
      to[2] = {state + r * head / 4, head};
      to[3] = {conv_state ? static_cast<const char*>(conv_state) + r * 6 * dim : nullptr, 6 * dim};
      if (overlaps(to, in)) return GDN_ERR_SHAPE;
    }
  }
  a.batch = batch; a.n_tok = n_tok;
  a.x = static_cast<const uint16_t*>(x); a.dt = dt; a.state = state; a.slot = slot;
  a.out = static_cast<uint16_t*>(out); a.snap = snapshots;
  a.conv_state = static_cast<uint16_t*>(conv_state);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_ssm_decode(a, s), s);
}

gdn_status gdn_rms_norm(const gdn_norm_shape* shape, int32_t n_rows, int32_t x_dtype, const void* x,
                        int64_t x_row_stride, int32_t res_dtype, const void* residual, int64_t res_row_stride,
                        void* residual_out, const void* gate, int64_t gate_row_stride, const float* weight, void* out,
                        int32_t code_dtype, void* codes, float* scales, void* stream) {
  if (!shape) return GDN_ERR_NULL;
  const int64_t d = shape->dim, rows = n_rows;
  if (d < 1 || shape->groups < 1 || d % shape->groups != 0 || n_rows < 0) return GDN_ERR_SHAPE;
  if (!(shape->eps >= 0.f) || !std::isfinite(shape->eps) || !std::isfinite(shape->weight_offset)) return GDN_ERR_SHAPE;
  const int64_t gd = d / shape->groups;
  if (d > 32768 || (shape->flags & ~GDN_NORM_GATE_FIRST)) return GDN_ERR_UNSUPPORTED;
  if (shape->groups > 1 && gd % 512 != 0 && (gd < 8 || gd > 512 || (gd & (gd - 1)) != 0)) return GDN_ERR_UNSUPPORTED;
  if (shape->weight_dim != d && shape->weight_dim != gd) return GDN_ERR_SHAPE;
  if (shape->scale_block != 0 && (shape->scale_block != 128 || d % 128 != 0)) return GDN_ERR_UNSUPPORTED;
  if (x_dtype != GDN_BF16 && x_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (residual && res_dtype != GDN_BF16 && res_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (codes && code_dtype != GDN_E4M3 && code_dtype != GDN_I8) return GDN_ERR_UNSUPPORTED;
  const int64_t xs = x_row_stride == 0 ? d : x_row_stride, rs = res_row_stride == 0 ? d : res_row_stride;
  const int64_t zs = gate_row_stride == 0 ? d : gate_row_stride;
  if (xs < d || rs < d || zs < d || xs > INT32_MAX || rs > INT32_MAX || zs > INT32_MAX) return GDN_ERR_SHAPE;
  if (n_rows == 0) return GDN_OK;
  if (!x || !codes != !scales || (residual_out && !residual)) return GDN_ERR_NULL;
  if (!out && !codes && !residual_out) return GDN_ERR_NULL;
  if ((shape->flags & GDN_NORM_GATE_FIRST) && !gate) return GDN_ERR_NULL;
  const int64_t xb = x_dtype == GDN_BF16 ? 2 : 4, rb = res_dtype == GDN_BF16 ? 2 : 4;
  const uintptr_t odd = (uintptr_t)x | (uintptr_t)gate | (uintptr_t)out, rodd = (uintptr_t)residual | (uintptr_t)residual_out;
  if (odd % xb != 0 || rodd % rb != 0 || ((uintptr_t)weight | (uintptr_t)scales) % 4 != 0) return GDN_ERR_SHAPE;
  // what is written overlaps nothing, but residual_out may be residual and out a dense x
  const int64_t scale_n = shape->scale_block ? d / 128 : 1;
  const Span in[] = {{x, ((rows - 1) * xs + d) * xb}, {residual, ((rows - 1) * rs + d) * rb},
                     {gate, ((rows - 1) * zs + d) * xb}, {weight, shape->weight_dim * 4}};
  const Span to[] = {{out, rows * d * xb, xs == d ? 0 : -1}, {residual_out, ((rows - 1) * rs + d) * rb, 1},
                     {codes, rows * d}, {scales, rows * scale_n * 4}};
  if (overlaps(to, in)) return GDN_ERR_SHAPE;
  if (!fits_grid(rows, d <= 512 ? 64 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024)) return GDN_ERR_SHAPE;
  gdn::NormArgs a{};
  a.dim = (int32_t)d; a.groups = shape->groups; a.group_dim = (int32_t)gd; a.scale_block = shape->scale_block;
  a.n_rows = n_rows; a.x_f32 = x_dtype == GDN_F32; a.res_f32 = res_dtype == GDN_F32;
  a.gate_first = (shape->flags & GDN_NORM_GATE_FIRST) != 0; a.codes_i8 = code_dtype == GDN_I8;
  a.eps = shape->eps; a.weight_offset = shape->weight_offset; a.weight_dim = shape->weight_dim;
  a.x = x; a.res = residual; a.gate = gate; a.x_stride = xs; a.res_stride = rs; a.gate_stride = zs;
  a.w = weight; a.out = out; a.res_out = residual_out; a.codes = static_cast<uint8_t*>(codes); a.scales = scales;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return finish_launch(gdn::launch_rms_norm(a, s), s);
}

}  // extern "C"
