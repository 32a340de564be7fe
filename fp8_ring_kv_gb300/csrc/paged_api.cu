// Host side of the paged cache: argument checks, workspace layout, RoPE
// tables, TMA descriptors and kernel launches.  See include/kvring_paged.h.
#include <cmath>
#include <cstring>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/kvring_paged.h"
#include "host.h"
#include "launch.h"
#include "paged.h"

using namespace kvring_dev;

static_assert(KVRING_DEVERR_SEQ == DEVERR_SEQ && KVRING_DEVERR_PAGE == DEVERR_PAGE, "error bits");
static_assert(KVRING_PAGED_MAX_SEQS == kPagedMaxSeqs && KVRING_PAGED_MAX_LEN == kPagedMaxLen, "limits");

struct kvring_paged {
  kvring_paged_config cfg;
  PagedView pv;               // layer 0
  CUtensorMap k_map, v_map;   // e4m3 rows of every layer, box {D, min(P, 32)}
  uint8_t* scratch;
  int device, sms;
};

namespace {

struct PagedLayout {
  size_t state, omega, rope[3], k_codes, v_codes, k_scale, v_scale, scratch, total;
};

bool check_config(const kvring_paged_config* c) {
  if (!c) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->layers < 1 || c->kv_heads < 1 || c->kv_heads > 128 || c->q_heads < 1 || c->q_heads > 1024) return false;
  if (c->q_heads % c->kv_heads) return false;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128) return false;
  if (c->n_pages < 1) return false;
  const long long blocks = (long long)c->layers * c->n_pages;   // < 2^62
  if (blocks >= (1ll << 31) || blocks * c->kv_heads * c->page_tokens >= (1ll << 31)) return false;
  if (c->in_dtype != KVRING_IN_BF16 && c->in_dtype != KVRING_IN_F16) return false;
  return rope_axes_ok(c->n_axes, c->axis_dims, c->pos_count, c->head_dim, c->rope_base);
}

PagedLayout layout_of(const kvring_paged_config* c) {
  PagedLayout L{};
  const size_t blocks = (size_t)c->layers * c->n_pages * c->kv_heads;
  const size_t codes = blocks * c->page_tokens * c->head_dim;
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
  L.k_codes = take(codes);
  L.v_codes = take(codes);
  L.k_scale = take(blocks * sizeof(float));
  L.v_scale = take(blocks * sizeof(float));
  L.scratch = take(paged_scratch_bytes(c->head_dim));
  L.total = off;
  return L;
}

bool encode_codes(CUtensorMap* m, void* codes, const kvring_paged_config& c) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t D = c.head_dim;
  const cuuint64_t dims[2] = {D, (cuuint64_t)c.layers * c.n_pages * c.kv_heads * c.page_tokens};
  const cuuint64_t strides[1] = {D};
  const cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)(c.page_tokens < 32 ? c.page_tokens : 32)};
  const cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the checks that both calls share; KVRING_OK also sets *pv and *pb
int check_batch(const kvring_paged* p, int32_t layer, const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs,
                int32_t n_tokens, const int32_t* table, int64_t table_stride, int32_t table_width, PagedView* pv,
                PagedBatch* pb) {
  if (!p || !seq_start || !kv_len || !table) return KVRING_ERR_INVALID_ARG;
  if (layer < 0 || layer >= p->cfg.layers) return KVRING_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_seqs > KVRING_PAGED_MAX_SEQS || n_tokens < 0 || n_tokens > (1 << 24))
    return KVRING_ERR_INVALID_ARG;
  if (table_width < 1 || table_stride < table_width ||
      (long long)table_width * p->cfg.page_tokens > KVRING_PAGED_MAX_LEN)
    return KVRING_ERR_INVALID_ARG;
  if (!aligned(seq_start, 4) || !aligned(kv_len, 4) || !aligned(table, 4)) return KVRING_ERR_MISALIGNED;
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev != p->device) return KVRING_ERR_INVALID_ARG;
  *pv = p->pv;
  const size_t blocks = (size_t)layer * p->cfg.n_pages * p->cfg.kv_heads;
  const size_t rows = blocks * p->cfg.page_tokens;
  pv->k_codes += rows * p->cfg.head_dim;
  pv->v_codes += rows * p->cfg.head_dim;
  pv->k_scale += blocks;
  pv->v_scale += blocks;
  pv->row0 = (long long)rows;
  *pb = PagedBatch{seq_start, kv_len, table, table_stride, n_seqs, n_tokens, table_width};
  return KVRING_OK;
}

bool stride_ok(int64_t stride, int heads, int D) {
  return stride >= (int64_t)heads * D && stride % 8 == 0 && stride < (1ll << 40);
}

}  // namespace

extern "C" {

size_t kvring_paged_workspace_bytes(const kvring_paged_config* cfg) {
  return check_config(cfg) ? layout_of(cfg).total : 0;
}

int kvring_paged_create(const kvring_paged_config* cfg, void* workspace, size_t workspace_bytes,
                        kvring_stream stream, kvring_paged** out) {
  if (!out) return KVRING_ERR_INVALID_ARG;
  *out = nullptr;
  if (!check_config(cfg) || !workspace) return KVRING_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return KVRING_ERR_MISALIGNED;
  const PagedLayout L = layout_of(cfg);
  if (workspace_bytes < L.total) return KVRING_ERR_WORKSPACE;
  int dev = 0, major = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (major != 10) return KVRING_ERR_NO_DEVICE;

  kvring_paged* p = new (std::nothrow) kvring_paged;
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
  pv.k_codes = ws + L.k_codes;
  pv.v_codes = ws + L.v_codes;
  pv.k_scale = reinterpret_cast<float*>(ws + L.k_scale);
  pv.v_scale = reinterpret_cast<float*>(ws + L.v_scale);
  pv.H = cfg->kv_heads;
  pv.QH = cfg->q_heads;
  pv.G = cfg->q_heads / cfg->kv_heads;
  pv.D = cfg->head_dim;
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
  if (e == cudaSuccess) e = cudaMemsetAsync(ws + L.k_codes, 0, L.scratch - L.k_codes, st);
  // pageable source: the copy is staged before the call returns
  if (e == cudaSuccess) e = cudaMemcpyAsync(ws + L.omega, om, sizeof(om), cudaMemcpyHostToDevice, st);
  for (int a = 0; e == cudaSuccess && a < cfg->n_axes; ++a)
    e = launch_paged_rope_table(reinterpret_cast<float2*>(ws + L.rope[a]), cfg->pos_min[a], cfg->pos_count[a],
                                cfg->axis_dims[a] / 2, reinterpret_cast<const double*>(ws + L.omega) + a * 64, st);
  if (e == cudaSuccess && (!encode_codes(&p->k_map, pv.k_codes, *cfg) || !encode_codes(&p->v_map, pv.v_codes, *cfg)))
    e = cudaErrorInvalidValue;
  if (e == cudaSuccess) e = prepare_paged_rows(pv.D);
  if (e == cudaSuccess) e = prepare_paged_tiles(pv.D);
  if (e != cudaSuccess) {
    delete p;
    return cuda_fail(e);
  }
  *out = p;
  return KVRING_OK;
}

int kvring_paged_append(kvring_paged* p, int32_t layer, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const int32_t* pos, const int32_t* seq_start, const int32_t* kv_len,
                        int32_t n_seqs, int32_t n_tokens, const int32_t* page_table, int64_t table_stride,
                        int32_t table_width, kvring_stream stream) {
  if (!k || !v || !pos) return KVRING_ERR_INVALID_ARG;
  PagedView pv;
  PagedBatch pb;
  const int s = check_batch(p, layer, seq_start, kv_len, n_seqs, n_tokens, page_table, table_stride, table_width, &pv,
                            &pb);
  if (s != KVRING_OK) return s;
  if (!stride_ok(k_stride, pv.H, pv.D) || !stride_ok(v_stride, pv.H, pv.D)) return KVRING_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4)) return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_tokens == 0) return KVRING_OK;
  const cudaError_t e = launch_paged_append(pv, pb, k, k_stride, v, v_stride, pos, p->cfg.in_dtype == KVRING_IN_F16,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_paged_attend(kvring_paged* p, int32_t layer, const void* q, int64_t q_stride, const int32_t* q_pos,
                        const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs, int32_t n_tokens,
                        int32_t max_new, const int32_t* page_table, int64_t table_stride, int32_t table_width,
                        int32_t causal, int32_t window, float scale, void* out, int64_t out_stride,
                        kvring_stream stream) {
  if (!q || !q_pos || !out) return KVRING_ERR_INVALID_ARG;
  PagedAttn a{};
  const int s = check_batch(p, layer, seq_start, kv_len, n_seqs, n_tokens, page_table, table_stride, table_width,
                            &a.pv, &a.pb);
  if (s != KVRING_OK) return s;
  if (!stride_ok(q_stride, a.pv.QH, a.pv.D) || !stride_ok(out_stride, a.pv.QH, a.pv.D)) return KVRING_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return KVRING_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || !std::isfinite(scale)) return KVRING_ERR_INVALID_ARG;
  if ((long long)n_tokens * a.pv.G > (1ll << 30)) return KVRING_ERR_INVALID_ARG;   // rows are 32-bit numbers
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(q_pos, 4)) return KVRING_ERR_MISALIGNED;
  if (n_seqs == 0 || n_tokens == 0) return KVRING_OK;
  if (max_new < 1 || max_new > n_tokens) return KVRING_ERR_INVALID_ARG;
  a.q = q;
  a.q_pos = q_pos;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale_log2 = (float)((scale > 0.0f ? (double)scale : 1.0 / std::sqrt((double)a.pv.D)) * 1.4426950408889634);
  if (!std::isfinite(a.scale_log2)) return KVRING_ERR_INVALID_ARG;
  a.causal = causal;
  a.window = window < KVRING_PAGED_MAX_LEN ? window : 0;   // wider than any sequence: none
  a.max_new = max_new;
  paged_carve_scratch(p->scratch, a.pv.D, &a);
  const cudaError_t e = launch_paged_attend(a, p->k_map, p->v_map, p->cfg.in_dtype == KVRING_IN_F16, p->sms,
                                            reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

int kvring_paged_destroy(kvring_paged* p) {
  delete p;
  return KVRING_OK;
}

int kvring_paged_layout(const kvring_paged* p, void** k_codes, void** v_codes, void** k_scales, void** v_scales,
                        void** state) {
  if (!p) return KVRING_ERR_INVALID_ARG;
  if (k_codes) *k_codes = p->pv.k_codes;
  if (v_codes) *v_codes = p->pv.v_codes;
  if (k_scales) *k_scales = p->pv.k_scale;
  if (v_scales) *v_scales = p->pv.v_scale;
  if (state) *state = p->pv.state;
  return KVRING_OK;
}

int kvring_paged_debug_state(const kvring_paged* p, kvring_stream stream, int32_t* err) {
  if (!p || !err) return KVRING_ERR_INVALID_ARG;
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaMemcpy(err, p->pv.state + PST_ERR, sizeof(*err), cudaMemcpyDeviceToHost);
  return e == cudaSuccess ? KVRING_OK : cuda_fail(e);
}

}  // extern "C"
