// latent_append and latent_read: rows into the paged latent cache and back.
//
// A token's row is by itself: x = (latent, rotated part), s = 2^k the smallest
// power of two with max |x| <= 448 s, codes e4m3(x / s).  A warp has the whole
// row, so the maximum is a warp's reduction and nothing is read twice.  A row
// with anything that is no number of the cache's range is marked by a scale of
// NaN and holds zeros: the attention's masked weights (zeros) then meet no NaN
// code, and the queries that see the token get their NaN through its score.
//
// What bounds it: the chain of loads token -> sequence -> page for few tokens (2.4 to
// 2.7 us warm, 9 cold); for many the bytes (3 (C + 64) a token, each way) behind such
// chains: 16,662 tokens of 512 + 64 appended in 15 us cold (1.9 TB/s), 92,383 rows
// read back in 34 (4.7 TB/s, 70% of a copy's rate).
#include "latent.h"
#include "launch.h"

namespace kvring_dev {

constexpr int kRowWarps = 8;
// Rows of a warp, their chains of loads side by side; one where there are few rows,
// whose warps all run at once.  Append, one and four rows (us, warm): 777 tokens 2.4
// and 3.2, 4,000 tokens 4.0 and 3.5, 9,600 tokens 6.7 and 4.6.  Read, one, two and four
// (cold): 92,000 rows 38, 34 and 36.
constexpr int kAppendRows = 4, kReadRows = 2, kFewRows = 2 * kRowWarps * 152;

// Where a packed row belongs.  page < 0: nowhere.
struct RowPlace {
  int page, off;
};

// Of rows tok0 .. tok0 + rows - 1 in lanes 0 .. rows - 1 (page -1 in the others): the
// sequence of the first is the last b with seq_start[b] <= tok0 (32 probes at a time),
// that of the others the same or, a few loads on, a later one; from there the page.
// Starts that decrease may lose sequences, never reach outside the call's arrays.
__device__ __forceinline__ RowPlace row_places(const PagedView& pv, const PagedBatch& pb, int tok0, int rows) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = pb.n_seqs;                             // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + lane * step;
    const bool le = i < lo + n && (i == lo || pb.seq_start[i] <= tok0);
    const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, le));
    const int nlo = lo + last * step;
    n = min(step, lo + n - nlo);
    lo = nlo;
  }
  RowPlace p = {-1, 0};
  if (lane >= rows) return p;
  const int tok = tok0 + lane;
  while (lo + 1 < pb.n_seqs && pb.seq_start[lo + 1] <= tok) ++lo;
  bool ok;
  const SeqInfo s = seq_info(pb, pv.p_shift, lo, ok);
  if (!ok || tok < s.s0 || tok >= s.s0 + s.n || s.n > s.len) return p;
  const int t = s.len - s.n + tok - s.s0;
  p.off = t & (pv.P - 1);
  p.page = pb.table[lo * pb.table_stride + (t >> pv.p_shift)];
  if (p.page < 0 || p.page >= pv.n_pages) {
    atomicOr(&pv.state[PST_ERR], DEVERR_PAGE);
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

template <typename T, int R>
__global__ void __launch_bounds__(32 * kRowWarps)
    latent_append_kernel(PagedView pv, PagedBatch pb, const T* latent, long long latent_stride, const T* rope,
                         long long rope_stride, const int32_t* pos) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  report_seqs(pv, pb);
  const int tok0 = (blockIdx.x * kRowWarps + warp) * R, rows = min(R, pb.n_tokens - tok0);
  if (rows <= 0) return;                                 // the whole warp
  // lane l: latent numbers 16 l .. 16 l + 15 of every row, and 16 of the rotated part
  // of row l / 4
  const bool mine = lane * 16 < pv.D;
  const int rr = lane >> 2, part = lane & 3;
  const bool turns = rr < rows;
  uint4 a[R][2], r0 = {}, r1 = {};
#pragma unroll
  for (int k = 0; k < R; ++k) {
    a[k][0] = a[k][1] = make_uint4(0, 0, 0, 0);
    if (mine && k < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(latent + (tok0 + k) * latent_stride) + 2 * lane;
      a[k][0] = src[0];
      a[k][1] = src[1];
    }
  }
  bool bad = false;
  float2 cs[8];
  if (turns) {
    const uint4* src = reinterpret_cast<const uint4*>(rope + (tok0 + rr) * rope_stride) + 2 * part;
    r0 = src[0];
    r1 = src[1];
    rope_load(pv, rope_lane(pv, part * 8), pos + (size_t)(tok0 + rr) * pv.n_axes, cs, bad);
  }
  const RowPlace at = row_places(pv, pb, tok0, rows);
  const int my_page = __shfl_sync(0xFFFFFFFFu, at.page, rr), my_off = __shfl_sync(0xFFFFFFFFu, at.off, rr);
  if (bad && turns && my_page >= 0) atomicOr(&pv.state[PST_ERR], DEVERR_POS_RANGE);
  // magnitudes by their bits: an infinity is above every number, a NaN above that
  float y[16];
  uint32_t ytop = 0;
  if (turns) {
    load8_f32<T>(r0, y);
    load8_f32<T>(r1, y + 8);
#pragma unroll
    for (int m = 0; m < 8; ++m) rope_pair(y[2 * m], y[2 * m + 1], cs[m].x, cs[m].y);
#pragma unroll
    for (int i = 0; i < 16; ++i) ytop = max(ytop, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  }
  ytop = max(ytop, __shfl_xor_sync(0xFFFFFFFFu, ytop, 1));
  ytop = max(ytop, __shfl_xor_sync(0xFFFFFFFFu, ytop, 2));
  const uint4 zero = make_uint4(0, 0, 0, 0);
  float my_inv = 0.0f;                                   // 0: not in range
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float x[16];
    load8_f32<T>(a[k][0], x);
    load8_f32<T>(a[k][1], x + 8);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(__reduce_max_sync(0xFFFFFFFFu, top), __shfl_sync(0xFFFFFFFFu, ytop, 4 * k));
    const float amax = __uint_as_float(top);
    float scale = kLatMinScale, inv = 1.0f / kLatMinScale;
    const bool in_range = amax <= 448.0f * kLatMaxScale; // false for a NaN
    if (in_range && amax > 448.0f * kLatMinScale) pow2_scale(amax, scale, inv);
    if (rr == k && in_range) my_inv = inv;
    const int page = __shfl_sync(0xFFFFFFFFu, at.page, k), off = __shfl_sync(0xFFFFFFFFu, at.off, k);
    if (page < 0) continue;
    const size_t row = ((size_t)page << pv.p_shift) + off;
    if (mine) *reinterpret_cast<uint4*>(pv.k_codes + row * (pv.D + kLatRope) + lane * 16) = in_range ? codes16(x, inv) : zero;
    if (lane == k) pv.k_scale[row] = in_range ? scale : __int_as_float(0x7FC00000);
  }
  if (turns && my_page >= 0) {
    const size_t row = ((size_t)my_page << pv.p_shift) + my_off;
    *reinterpret_cast<uint4*>(pv.k_codes + row * (pv.D + kLatRope) + pv.D + part * 16) = my_inv > 0.0f ? codes16(y, my_inv) : zero;
  }
}

template <typename T>
__device__ __forceinline__ void read16(const uint4& codes, float scale, T* dst) {
  float x[16];
  dequant16_scaled(codes, scale, x);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T, int R>
__global__ void __launch_bounds__(32 * kRowWarps)
    latent_read_kernel(PagedView pv, PagedBatch pb, T* out, long long out_stride) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  report_seqs(pv, pb);
  const int tok0 = (blockIdx.x * kRowWarps + warp) * R, rows = min(R, pb.n_tokens - tok0);
  if (rows <= 0) return;
  const RowPlace at = row_places(pv, pb, tok0, rows);
  const bool mine = lane * 16 < pv.D;
  const int rr = lane >> 2, part = lane & 3;             // of the rotated parts, four lanes a row
  const int my_page = __shfl_sync(0xFFFFFFFFu, at.page, rr), my_off = __shfl_sync(0xFFFFFFFFu, at.off, rr);
  const bool turns = rr < R && my_page >= 0;
  const size_t my_row = ((size_t)max(my_page, 0) << pv.p_shift) + my_off;
  const int W = pv.D + kLatRope;
  uint4 c[R], r = {};
  float my_scale = 0.0f;
  if (turns) {
    my_scale = pv.k_scale[my_row];
    r = *reinterpret_cast<const uint4*>(pv.k_codes + my_row * W + pv.D + part * 16);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int page = __shfl_sync(0xFFFFFFFFu, at.page, k), off = __shfl_sync(0xFFFFFFFFu, at.off, k);
    c[k] = make_uint4(0, 0, 0, 0);
    if (mine && page >= 0)
      c[k] = *reinterpret_cast<const uint4*>(pv.k_codes + (((size_t)page << pv.p_shift) + off) * W + lane * 16);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const float scale = __shfl_sync(0xFFFFFFFFu, my_scale, 4 * k);
    const bool placed = __shfl_sync(0xFFFFFFFFu, at.page, k) >= 0;
    if (mine && placed) read16<T>(c[k], scale, out + (tok0 + k) * out_stride + lane * 16);
  }
  if (turns) read16<T>(r, my_scale, out + (tok0 + rr) * out_stride + pv.D + part * 16);
}

template <typename T, int R>
static cudaError_t append_t(const PagedView& pv, const PagedBatch& pb, const void* latent, long long latent_stride,
                            const void* rope, long long rope_stride, const int32_t* pos, cudaStream_t st) {
  constexpr int per = kRowWarps * R;
  const dim3 grid((unsigned)((pb.n_tokens + per - 1) / per)), block(32 * kRowWarps);
  return launch_pdl(latent_append_kernel<T, R>, grid, block, 0, st, pv, pb, static_cast<const T*>(latent), latent_stride,
                    static_cast<const T*>(rope), rope_stride, pos);
}

cudaError_t launch_latent_append(const PagedView& pv, const PagedBatch& pb, const void* latent, long long latent_stride,
                                 const void* rope, long long rope_stride, const int32_t* pos, bool f16,
                                 cudaStream_t st) {
  const auto fn = pb.n_tokens <= kFewRows ? (f16 ? append_t<__half, 1> : append_t<__nv_bfloat16, 1>)
                                          : (f16 ? append_t<__half, kAppendRows> : append_t<__nv_bfloat16, kAppendRows>);
  return fn(pv, pb, latent, latent_stride, rope, rope_stride, pos, st);
}

template <typename T, int R>
static cudaError_t read_t(const PagedView& pv, const PagedBatch& pb, void* out, long long out_stride, cudaStream_t st) {
  constexpr int per = kRowWarps * R;
  const dim3 grid((unsigned)((pb.n_tokens + per - 1) / per)), block(32 * kRowWarps);
  return launch_pdl(latent_read_kernel<T, R>, grid, block, 0, st, pv, pb, static_cast<T*>(out), out_stride);
}

cudaError_t launch_latent_read(const PagedView& pv, const PagedBatch& pb, void* out, long long out_stride, bool f16,
                               cudaStream_t st) {
  const auto fn = pb.n_tokens <= kFewRows ? (f16 ? read_t<__half, 1> : read_t<__nv_bfloat16, 1>)
                                          : (f16 ? read_t<__half, kReadRows> : read_t<__nv_bfloat16, kReadRows>);
  return fn(pv, pb, out, out_stride, st);
}

}  // namespace kvring_dev
