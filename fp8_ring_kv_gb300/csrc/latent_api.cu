// Host side of the latent cache: argument checks, workspace layout, RoPE
// tables, TMA descriptors and kernel launches.  See include/kvring_latent.h.
#include <cmath>
#include <cstring>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/kvring_latent.h"
#include "host.h"
#include "latent.h"
#include "launch.h"

using namespace kvring_dev;

static_assert(KVRING_LATENT_ROPE == kLatRope && KVRING_LATENT_HEAD == kLatHead, "sizes");

struct kvring_latent {
  kvring_latent_config cfg;
  PagedView pv;               // layer 0
  CUtensorMap c_map, r_map;   // code rows of every layer, boxes {128, P} and {64, P}
  uint8_t* scratch;
  int device, sms;
};

namespace {

struct LatentLayout {
  size_t state, omega, rope[3], codes, scales, scratch, total;
};

bool check_config(const kvring_latent_config* c) {
  if (!c) return false;
  if (c->latent_dim < 128 || c->latent_dim > kLatMax || c->latent_dim % 128) return false;
  if (c->layers < 1 || c->q_heads < 1 || c->q_heads > 256) return false;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return false;
  if (c->n_pages < 1) return false;
  const long long blocks = (long long)c->layers * c->n_pages;   // < 2^62
  if (blocks >= (1ll << 31) || blocks * c->page_tokens >= (1ll << 31)) return false;
  if (c->in_dtype != KVRING_IN_BF16 && c->in_dtype != KVRING_IN_F16) return false;
  return rope_axes_ok(c->n_axes, c->axis_dims, c->pos_count, kLatRope, c->rope_base);
}

LatentLayout layout_of(const kvring_latent_config* c) {
  LatentLayout L{};
  const size_t rows = (size_t)c->layers * c->n_pages * c->page_tokens;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 1024);
    return at;
  };
  L.state = take(PST_WORDS * sizeof(int32_t));
  L.omega = take(3 * 64 * sizeof(double));
  for (int a = 0; a < 3; ++a)
    L.rope[a] = take(a < c->n_axes ? (size_t)c->pos_count[a] * (c->axis_dims[a] / 2) * sizeof(float2) : 0);
  L.codes = take(rows * (c->latent_dim + kLatRope));
  L.scales = take(rows * sizeof(float));
  L.scratch = take(latent_scratch_bytes(c->latent_dim));
  L.total = off;
  return L;
}

bool encode_rows(CUtensorMap* m, void* codes, const kvring_latent_config& c, int width) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t W = c.latent_dim + kLatRope;
  const cuuint64_t dims[2] = {W, (cuuint64_t)c.layers * c.n_pages * c.page_tokens};
  const cuuint64_t strides[1] = {W};
  const cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)c.page_tokens};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 16-bit rows [heads][n][width] (heads 0: [n][width]), boxes of 64 numbers of
// ``rows`` rows.  A tensor of no rows has none to read: one, of which nothing is read.
bool encode_heads(CUtensorMap* m, const void* base, bool f16, int width, int heads, int n, long long token,
                  long long head, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  // a stride that is not used may be anything; the encoder wants a positive one
  const cuuint64_t strides[2] = {(cuuint64_t)(token > 0 ? token : width) * 2, (cuuint64_t)(head > 0 ? head : width) * 2};
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)(n > 0 ? n : 1), (cuuint64_t)heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, heads > 0 ? 3 : 2,
             const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the checks that all calls share
int check_call(const kvring_latent* p, const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs,
               int32_t n_tokens) {
  if (!p || !seq_start || !kv_len) return KVRING_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_seqs > KVRING_PAGED_MAX_SEQS || n_tokens < 0 || n_tokens > (1 << 24))
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(seq_start, 4) || !aligned(kv_len, 4)) return KVRING_ERR_MISALIGNED;
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  return dev == p->device ? KVRING_OK : KVRING_ERR_INVALID_ARG;
}

// and those of the calls on the pages; KVRING_OK also sets *pv and *pb
int check_pages(const kvring_latent* p, int32_t layer, const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs,
                int32_t n_tokens, const int32_t* table, int64_t table_stride, int32_t table_width, PagedView* pv,
                PagedBatch* pb) {
  const int s = check_call(p, seq_start, kv_len, n_seqs, n_tokens);
  if (s != KVRING_OK) return s;
  if (!table || layer < 0 || layer >= p->cfg.layers) return KVRING_ERR_INVALID_ARG;
  if (table_width < 1 || table_stride < table_width ||
      (long long)table_width * p->cfg.page_tokens > KVRING_PAGED_MAX_LEN)
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(table, 4)) return KVRING_ERR_MISALIGNED;
  *pv = p->pv;
  const size_t rows = (size_t)layer * p->cfg.n_pages * p->cfg.page_tokens;
  pv->k_codes += rows * (p->cfg.latent_dim + kLatRope);
  pv->k_scale += rows;
  pv->row0 = (long long)rows;
  *pb = PagedBatch{seq_start, kv_len, table, table_stride, n_seqs, n_tokens, table_width};
  return KVRING_OK;
}

bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride < (1ll << 40); }

// Rows of [n][heads][width]: neither heads nor tokens overlap, one of the two
// being the outer one.  A stride that is not used (one token, one head) may be anything.
bool strides_ok(Strides s, int64_t n, int64_t heads, int64_t width) {
  if (s.token < 0 || s.head < 0 || s.token % 8 || s.head % 8 || s.token >= (1ll << 40) || s.head >= (1ll << 40))
    return false;
  if (n <= 1) return heads <= 1 || s.head >= width;
  if (heads <= 1) return s.token >= width;
  return (s.head >= width && s.token >= (heads - 1) * s.head + width) ||
         (s.token >= width && s.head >= (n - 1) * s.token + width);
}

int check_attend(const kvring_latent* p, int32_t n_tokens, int32_t max_new, int32_t causal, int32_t window, float scale,
                 PagedAttn* a) {
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return KVRING_ERR_INVALID_ARG;
  if (!(scale >= 0x1p-100f && scale <= 0x1p100f)) return KVRING_ERR_INVALID_ARG;
  if ((long long)n_tokens * p->cfg.q_heads > (1ll << 30)) return KVRING_ERR_INVALID_ARG;   // rows are 32-bit numbers
  if (n_tokens > 0 && (max_new < 1 || max_new > n_tokens)) return KVRING_ERR_INVALID_ARG;
  a->scale_log2 = (float)((double)scale * 1.4426950408889634);
  a->causal = causal;
  a->window = window < KVRING_PAGED_MAX_LEN ? window : 0;   // wider than any sequence: none
  a->max_new = max_new;
  return KVRING_OK;
}

}  // namespace

extern "C" {

size_t kvring_latent_workspace_bytes(const kvring_latent_config* cfg) {
  return check_config(cfg) ? layout_of(cfg).total : 0;
}

int kvring_latent_create(const kvring_latent_config* cfg, void* workspace, size_t workspace_bytes,
                         kvring_stream stream, kvring_latent** out) {
  if (!out) return KVRING_ERR_INVALID_ARG;
  *out = nullptr;
  if (!check_config(cfg) || !workspace) return KVRING_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return KVRING_ERR_MISALIGNED;
  const LatentLayout L = layout_of(cfg);
  if (workspace_bytes < L.total) return KVRING_ERR_WORKSPACE;
  int dev = 0, major = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (major != 10) return KVRING_ERR_NO_DEVICE;

  kvring_latent* p = new (std::nothrow) kvring_latent;
  if (!p) return KVRING_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  p->cfg = *cfg;
  p->device = dev;
  p->sms = sms;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PagedView& pv = p->pv;
  pv.state = reinterpret_cast<int32_t*>(ws + L.state);
  int pair_off = 0;
  for (int a = 0; a < 3; ++a) {
    const bool on = a < cfg->n_axes;
    pv.rope[a] = on ? reinterpret_cast<const float2*>(ws + L.rope[a]) : nullptr;
    pv.pos_min[a] = on ? cfg->pos_min[a] : 0;
    pv.pos_count[a] = on ? cfg->pos_count[a] : 1;
    pv.axis_pairs[a] = on ? cfg->axis_dims[a] / 2 : 0;
    pv.pair_off[a] = pair_off;
    if (on) pair_off += cfg->axis_dims[a] / 2;
  }
  pv.k_codes = ws + L.codes;
  pv.k_scale = reinterpret_cast<float*>(ws + L.scales);
  pv.H = 1;
  pv.QH = pv.G = cfg->q_heads;
  pv.D = cfg->latent_dim;
  pv.P = cfg->page_tokens;
  while ((1 << pv.p_shift) < pv.P) ++pv.p_shift;
  pv.n_pages = cfg->n_pages;
  pv.n_axes = cfg->n_axes;
  p->scratch = ws + L.scratch;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double om[3 * 64] = {};
  for (int a = 0; a < cfg->n_axes; ++a)
    for (int j = 0; j < cfg->axis_dims[a] / 2; ++j) om[a * 64 + j] = omega(cfg->rope_base, cfg->axis_dims[a], j);
  e = cudaMemsetAsync(ws + L.state, 0, L.omega - L.state, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws + L.codes, 0, L.scratch - L.codes, st);
  // pageable source: the copy is staged before the call returns
  if (e == cudaSuccess) e = cudaMemcpyAsync(ws + L.omega, om, sizeof(om), cudaMemcpyHostToDevice, st);
  for (int a = 0; e == cudaSuccess && a < cfg->n_axes; ++a)
    e = launch_paged_rope_table(reinterpret_cast<float2*>(ws + L.rope[a]), cfg->pos_min[a], cfg->pos_count[a],
                                cfg->axis_dims[a] / 2, reinterpret_cast<const double*>(ws + L.omega) + a * 64, st);
  if (e == cudaSuccess &&
      (!encode_rows(&p->c_map, pv.k_codes, *cfg, 128) || !encode_rows(&p->r_map, pv.k_codes, *cfg, kLatRope)))
    e = cudaErrorInvalidValue;
  if (e == cudaSuccess) e = prepare_latent_attend();
  if (e == cudaSuccess) e = prepare_latent_expanded();
  if (e != cudaSuccess) {
    delete p;
    return cuda_fail(e);
  }
  *out = p;
  return KVRING_OK;
}

int kvring_latent_append(kvring_latent* p, int32_t layer, const void* latent, int64_t latent_stride,
                         const void* k_rope, int64_t rope_stride, const int32_t* pos, const int32_t* seq_start,
                         const int32_t* kv_len, int32_t n_seqs, int32_t n_tokens, const int32_t* page_table,
                         int64_t table_stride, int32_t table_width, kvring_stream stream) {
  if (!latent || !k_rope || !pos) return KVRING_ERR_INVALID_ARG;
  PagedView pv;
  PagedBatch pb;
  const int s = check_pages(p, layer, seq_start, kv_len, n_seqs, n_tokens, page_table, table_stride, table_width, &pv,
                            &pb);
  if (s != KVRING_OK) return s;
  if (!stride_ok(latent_stride, pv.D) || !stride_ok(rope_stride, kLatRope)) return KVRING_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(k_rope, 16) || !aligned(pos, 4)) return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_tokens == 0) return KVRING_OK;
  const cudaError_t e = launch_latent_append(pv, pb, latent, latent_stride, k_rope, rope_stride, pos,
                                             p->cfg.in_dtype == KVRING_IN_F16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_latent_read(kvring_latent* p, int32_t layer, const int32_t* seq_start, const int32_t* kv_len,
                       int32_t n_seqs, int32_t n_rows, const int32_t* page_table, int64_t table_stride,
                       int32_t table_width, void* out, int64_t out_stride, kvring_stream stream) {
  if (!out) return KVRING_ERR_INVALID_ARG;
  PagedView pv;
  PagedBatch pb;
  const int s = check_pages(p, layer, seq_start, kv_len, n_seqs, n_rows, page_table, table_stride, table_width, &pv,
                            &pb);
  if (s != KVRING_OK) return s;
  if (!stride_ok(out_stride, pv.D + kLatRope)) return KVRING_ERR_INVALID_ARG;
  if (!aligned(out, 16)) return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_rows == 0) return KVRING_OK;
  const cudaError_t e = launch_latent_read(pv, pb, out, out_stride, p->cfg.in_dtype == KVRING_IN_F16,
                                           reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_latent_attend(kvring_latent* p, int32_t layer, const void* q_latent, int64_t q_latent_token,
                         int64_t q_latent_head, const void* q_rope, int64_t q_rope_token, int64_t q_rope_head,
                         const int32_t* q_pos, const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs,
                         int32_t n_tokens, int32_t max_new, const int32_t* page_table, int64_t table_stride,
                         int32_t table_width, int32_t causal, int32_t window, float scale, void* out,
                         int64_t out_token, int64_t out_head, kvring_stream stream) {
  if (!q_latent || !q_rope || !q_pos || !out) return KVRING_ERR_INVALID_ARG;
  LatentAttn la{};
  PagedAttn& a = la.a;
  int s = check_pages(p, layer, seq_start, kv_len, n_seqs, n_tokens, page_table, table_stride, table_width, &a.pv,
                      &a.pb);
  if (s == KVRING_OK) s = check_attend(p, n_tokens, max_new, causal, window, scale, &a);
  if (s != KVRING_OK) return s;
  la.q = {q_latent_token, q_latent_head};
  la.qr = {q_rope_token, q_rope_head};
  la.o = {out_token, out_head};
  if (!strides_ok(la.q, n_tokens, a.pv.G, a.pv.D) || !strides_ok(la.qr, n_tokens, a.pv.G, kLatRope) ||
      !strides_ok(la.o, n_tokens, a.pv.G, a.pv.D))
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(out, 16) || !aligned(q_pos, 4))
    return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_tokens == 0) return KVRING_OK;
  a.q = q_latent;
  a.q_pos = q_pos;
  a.out = out;
  la.q_rope = q_rope;
  la.code_rows = p->cfg.layers * p->cfg.n_pages * p->cfg.page_tokens;
  latent_carve_scratch(p->scratch, kLatRows, a.pv.D, &a);
  const cudaError_t e = launch_latent_attend(la, p->c_map, p->r_map, p->cfg.in_dtype == KVRING_IN_F16, p->sms,
                                             reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_latent_attend_expanded(kvring_latent* p, const void* q, int64_t q_token, int64_t q_head, const void* k,
                                  int64_t k_token, int64_t k_head, const void* k_rope, int64_t k_rope_token,
                                  const void* v, int64_t v_token, int64_t v_head, int32_t n_keys, const int32_t* q_pos,
                                  const int32_t* seq_start, const int32_t* kv_start, const int32_t* kv_len,
                                  int32_t n_seqs, int32_t n_tokens, int32_t max_new, int32_t causal, int32_t window,
                                  float scale, void* out, int64_t out_token, int64_t out_head, kvring_stream stream) {
  if (!q || !q_pos || !kv_start || !out) return KVRING_ERR_INVALID_ARG;
  if (n_keys == 0) k = v = k_rope = q;     // not read
  if (!k || !k_rope || !v) return KVRING_ERR_INVALID_ARG;
  ExpandedAttn xa{};
  PagedAttn& a = xa.a;
  int s = check_call(p, seq_start, kv_len, n_seqs, n_tokens);
  if (scale == 0.0f) scale = (float)(1.0 / std::sqrt((double)(kLatHead + kLatRope)));
  if (s == KVRING_OK) s = check_attend(p, n_tokens, max_new, causal, window, scale, &a);
  if (s != KVRING_OK) return s;
  const int heads = p->cfg.q_heads;
  xa.q = {q_token, q_head};
  xa.o = {out_token, out_head};
  xa.v = v;
  xa.v_token = v_token;
  xa.v_head = v_head;
  xa.n_keys = n_keys;
  if (n_keys < 0 || n_keys > (1 << 30)) return KVRING_ERR_INVALID_ARG;
  if (!strides_ok(xa.q, n_tokens, heads, kLatHead + kLatRope) || !strides_ok(xa.o, n_tokens, heads, kLatHead) ||
      !strides_ok({k_token, k_head}, n_keys, heads, kLatHead) || !strides_ok({v_token, v_head}, n_keys, heads, kLatHead) ||
      !stride_ok(k_rope_token, kLatRope))
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(k_rope, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(q_pos, 4) || !aligned(kv_start, 4))
    return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_tokens == 0) return KVRING_OK;
  a.pv = p->pv;
  a.pv.H = heads;
  a.pv.G = 1;
  a.pv.D = kLatHead;
  a.pv.p_shift = 22;                       // one "page" holds the longest sequence
  static_assert(KVRING_PAGED_MAX_LEN == 1 << 22, "a sequence's keys");
  a.pb = PagedBatch{seq_start, kv_len, kv_start, 1, n_seqs, n_tokens, 1};
  a.q = q;
  a.q_pos = q_pos;
  a.out = out;
  latent_carve_scratch(p->scratch, kTilesRows, kLatHead, &a);
  CUtensorMap tmK, tmV, tmR;
  const bool f16 = p->cfg.in_dtype == KVRING_IN_F16;
  if (!encode_heads(&tmK, k, f16, kLatHead, heads, n_keys, k_token, k_head, 128) ||
      !encode_heads(&tmV, v, f16, kLatHead, heads, n_keys, v_token, v_head, 64) ||
      !encode_heads(&tmR, k_rope, f16, kLatRope, 0, n_keys, k_rope_token, 0, 128))
    return cuda_fail(cudaErrorInvalidValue);
  const cudaError_t e = launch_latent_expanded(xa, tmK, tmR, tmV, f16, p->sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_latent_destroy(kvring_latent* p) {
  delete p;
  return KVRING_OK;
}

int kvring_latent_layout(const kvring_latent* p, void** codes, void** scales, void** state) {
  if (!p) return KVRING_ERR_INVALID_ARG;
  if (codes) *codes = p->pv.k_codes;
  if (scales) *scales = p->pv.k_scale;
  if (state) *state = p->pv.state;
  return KVRING_OK;
}

int kvring_latent_debug_state(const kvring_latent* p, kvring_stream stream, int32_t* err) {
  if (!p || !err) return KVRING_ERR_INVALID_ARG;
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaMemcpy(err, p->pv.state + PST_ERR, sizeof(*err), cudaMemcpyDeviceToHost);
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

}  // extern "C"
