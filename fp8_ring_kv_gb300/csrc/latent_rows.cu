// latent_append and latent_read: rows into the paged latent cache and back.
//
// A token's row is by itself: x = (latent, rotated part), s = 2^k the smallest
// power of two with max |x| <= 448 s, codes e4m3(x / s).  A warp has the whole
// row, so the maximum is a warp's reduction and nothing is read twice.  A row
// with anything that is no number of the cache's range is marked by a scale of
// NaN and holds zeros: the attention's masked weights (zeros) then meet no NaN
// code, and the queries that see the token get their NaN through its score.
//
// What bounds it: bytes for many tokens (3 (C + 64) per token), the chain of
// loads token -> sequence -> page for few.
#include "latent.h"
#include "launch.h"

namespace kvring_dev {

constexpr int kRowWarps = 8;

// Where a packed row belongs.  page < 0: nowhere.
struct RowPlace {
  int page, off;
};

// The sequence of row ``tok``: the last b with seq_start[b] <= tok (a warp, 32
// probes at a time), and from there its page.  Starts that decrease may lose
// sequences, never reach outside the call's arrays.
__device__ __forceinline__ RowPlace row_place(const PagedView& pv, const PagedBatch& pb, int tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = pb.n_seqs;                             // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + lane * step;
    const bool le = i < lo + n && (i == lo || pb.seq_start[i] <= tok);
    const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, le));
    const int nlo = lo + last * step;
    n = min(step, lo + n - nlo);
    lo = nlo;
  }
  bool ok;
  const SeqInfo s = seq_info(pb, pv.p_shift, lo, ok);
  RowPlace p = {-1, 0};
  if (!ok || tok < s.s0 || tok >= s.s0 + s.n || s.n > s.len) return p;
  const int t = s.len - s.n + tok - s.s0;
  p.off = t & (pv.P - 1);
  p.page = pb.table[lo * pb.table_stride + (t >> pv.p_shift)];
  if (p.page < 0 || p.page >= pv.n_pages) {
    if (lane == 0) atomicOr(&pv.state[PST_ERR], DEVERR_PAGE);
    p.page = -1;
  }
  return p;
}

// The sequences that are left out, flagged by the first block.
__device__ __forceinline__ void report_seqs(const PagedView& pv, const PagedBatch& pb) {
  if (blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < pb.n_seqs; b += blockDim.x) {
    bool ok;
    const SeqInfo s = seq_info(pb, pv.p_shift, b, ok);
    if (!ok || s.n > s.len) atomicOr(&pv.state[PST_ERR], DEVERR_SEQ);
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps)
    latent_append_kernel(PagedView pv, PagedBatch pb, const T* latent, long long latent_stride, const T* rope,
                         long long rope_stride, const int32_t* pos) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  report_seqs(pv, pb);
  const int tok = blockIdx.x * kRowWarps + warp;
  if (tok >= pb.n_tokens) return;                        // the whole warp
  // lane l: latent numbers 16 l .. 16 l + 15; lanes 0-3 also 16 of the rotated part
  const bool mine = lane * 16 < pv.D, turns = lane < kLatRope / 16;
  uint4 a0 = {}, a1 = {}, r0 = {}, r1 = {};
  if (mine) {
    const uint4* src = reinterpret_cast<const uint4*>(latent + tok * latent_stride) + 2 * lane;
    a0 = src[0];
    a1 = src[1];
  }
  bool bad = false;
  float2 cs[8];
  if (turns) {
    const uint4* src = reinterpret_cast<const uint4*>(rope + tok * rope_stride) + 2 * lane;
    r0 = src[0];
    r1 = src[1];
  }
  const RowPlace at = row_place(pv, pb, tok);
  if (at.page < 0) return;
  float x[16], y[16];
  load8_f32<T>(a0, x);
  load8_f32<T>(a1, x + 8);
  load8_f32<T>(r0, y);
  load8_f32<T>(r1, y + 8);
  if (turns) {
    rope_load(pv, rope_lane(pv, lane * 8), pos + (size_t)tok * pv.n_axes, cs, bad);
#pragma unroll
    for (int m = 0; m < 8; ++m) rope_pair(y[2 * m], y[2 * m + 1], cs[m].x, cs[m].y);
  }
  if (bad) atomicOr(&pv.state[PST_ERR], DEVERR_POS_RANGE);
  // magnitudes by their bits: an infinity is above every number, a NaN above that
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    top = max(top, max(__float_as_uint(x[i]) & 0x7FFFFFFFu, __float_as_uint(y[i]) & 0x7FFFFFFFu));
  const float amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, top));
  float scale = kLatMinScale, inv = 1.0f / kLatMinScale;
  const bool in_range = amax <= 448.0f * kLatMaxScale;   // false for a NaN
  if (in_range && amax > 448.0f * kLatMinScale) pow2_scale(amax, scale, inv);
  const size_t row = ((size_t)at.page << pv.p_shift) + at.off;
  uint8_t* codes = pv.k_codes + row * (pv.D + kLatRope);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (mine) *reinterpret_cast<uint4*>(codes + lane * 16) = in_range ? codes16(x, inv) : zero;
  if (turns) *reinterpret_cast<uint4*>(codes + pv.D + lane * 16) = in_range ? codes16(y, inv) : zero;
  if (lane == 0) pv.k_scale[row] = in_range ? scale : __int_as_float(0x7FC00000);
}

// Rows per warp: their chains of loads side by side.
constexpr int kReadRows = 4;

template <typename T>
__device__ __forceinline__ void read16(const uint8_t* src, float scale, T* dst) {
  float x[16];
  dequant16_scaled(*reinterpret_cast<const uint4*>(src), scale, x);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps)
    latent_read_kernel(PagedView pv, PagedBatch pb, T* out, long long out_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  report_seqs(pv, pb);
  const int tok0 = (blockIdx.x * kRowWarps + warp) * kReadRows;
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    const int tok = tok0 + k;
    if (tok >= pb.n_tokens) break;
    const RowPlace at = row_place(pv, pb, tok);
    if (at.page < 0) continue;
    const size_t row = ((size_t)at.page << pv.p_shift) + at.off;
    const float scale = pv.k_scale[row];
    const uint8_t* codes = pv.k_codes + row * (pv.D + kLatRope);
    T* dst = out + tok * out_stride;
    if (lane * 16 < pv.D) read16<T>(codes + lane * 16, scale, dst + lane * 16);
    if (lane < kLatRope / 16) read16<T>(codes + pv.D + lane * 16, scale, dst + pv.D + lane * 16);
  }
}

template <typename T>
static cudaError_t append_t(const PagedView& pv, const PagedBatch& pb, const void* latent, long long latent_stride,
                            const void* rope, long long rope_stride, const int32_t* pos, cudaStream_t st) {
  const unsigned blocks = (unsigned)((pb.n_tokens + kRowWarps - 1) / kRowWarps);
  return launch_pdl(latent_append_kernel<T>, dim3(blocks), dim3(32 * kRowWarps), 0, st, pv, pb,
                    static_cast<const T*>(latent), latent_stride, static_cast<const T*>(rope), rope_stride, pos);
}

cudaError_t launch_latent_append(const PagedView& pv, const PagedBatch& pb, const void* latent, long long latent_stride,
                                 const void* rope, long long rope_stride, const int32_t* pos, bool f16,
                                 cudaStream_t st) {
  return f16 ? append_t<__half>(pv, pb, latent, latent_stride, rope, rope_stride, pos, st)
             : append_t<__nv_bfloat16>(pv, pb, latent, latent_stride, rope, rope_stride, pos, st);
}

cudaError_t launch_latent_read(const PagedView& pv, const PagedBatch& pb, void* out, long long out_stride, bool f16,
                               cudaStream_t st) {
  constexpr int per = kRowWarps * kReadRows;
  const dim3 grid((unsigned)((pb.n_tokens + per - 1) / per)), block(32 * kRowWarps);
  return f16 ? launch_pdl(latent_read_kernel<__half>, grid, block, 0, st, pv, pb, static_cast<__half*>(out), out_stride)
             : launch_pdl(latent_read_kernel<__nv_bfloat16>, grid, block, 0, st, pv, pb,
                          static_cast<__nv_bfloat16*>(out), out_stride);
}

}  // namespace kvring_dev
