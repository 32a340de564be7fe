// Rows of the paged attention whose pages' V scales lie far apart.
//
// The kernels' weights are fp16 numbers that carry their page's V scale, with the
// row's largest such product near the top of fp16.  Where one page's scale is 2^e
// times another's, the other's weights lie up to 2^e lower there, and are rounded to
// 2^-25 2^e / 2^8 (2^6 in the tile kernel) of the row's largest weight: with e up to
// kScaleSpan, 2^-19 and 2^-17, and nothing to speak of for the values that trained
// models give.  A piece of an item whose scales differ by more (or are beyond
// 2^+-kScaleTop, which leaves fp32 room to join the pieces) is computed once more by
// exact_row, in fp32 with the scales where the formula has them: a warp a row, a key
// after the other.  Slow (some 60 instructions a key and row) and right: an output
// channel keeps its precision whatever the other pages hold, seen or not.
#pragma once
#include "paged.h"

namespace kvring_dev {

constexpr int kScaleSpan = 14, kScaleTop = 40;

// The smallest and the largest exponent of the scales that a lane has met; zeros (and
// what is no scale) do not count.
struct ScaleSpan {
  int top = -1024, low = 1024;
  __device__ __forceinline__ void add(float s) {
    const int e = (int)(__float_as_uint(s) >> 23) - 127;
    if (s > 0.0f && s < INFINITY) {
      top = max(top, e);
      low = min(low, e);
    }
  }
  // of the warp's lanes together
  __device__ __forceinline__ bool far_apart() const {
    const int t = __reduce_max_sync(0xFFFFFFFFu, top), l = __reduce_min_sync(0xFFFFFFFFu, low);
    return t >= l && (t - l > kScaleSpan || t > kScaleTop || l < -kScaleTop);
  }
};

// Row ``row`` (token row / G of sequence b's new ones, key head h) over the keys
// [k0, k1) of those that it sees; one warp.  dst: the output row, or null and the
// results to o [D] (unnormalised) and *ml (maximum of the scores and ``head``, the
// log2 of a largest weight in the kernel's other pieces; sum).
template <int D, typename T>
__device__ __noinline__ void exact_row(const PagedAttn& a, int b, int s0, int n, int len, int h, int row, int k0, int k1,
                                       T* dst, float* o_at, float2* ml, float head) {
  constexpr int V = D / 32;                              // channels of a lane
  const int lane = threadIdx.x & 31;
  const int i = row / a.pv.G, at = len - n + i;
  k1 = min(k1, a.causal ? at + 1 : len);
  if (a.window > 0) k0 = max(k0, at - a.window + 1);
  float x[V], o[V], m = -INFINITY, l = 0.0f;
  const T* src = static_cast<const T*>(a.q) + (s0 + i) * a.q_stride + (size_t)(h * a.pv.G + row - i * a.pv.G) * D + lane * V;
  bool bad = false;
#pragma unroll
  for (int p = 0; p < V / 2; ++p) {
    const float2 cs = rope_cs(a.pv, a.q_pos + (size_t)(s0 + i) * a.pv.n_axes, lane * (V / 2) + p, bad);
    const float2 y = rope_query((float)src[2 * p], (float)src[2 * p + 1], cs);
    x[2 * p] = y.x;
    x[2 * p + 1] = y.y;
    o[2 * p] = o[2 * p + 1] = 0.0f;
  }
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    int pg = a.pb.table[b * a.pb.table_stride + (k >> a.pv.p_shift)];
    if (pg < 0 || pg >= a.pv.n_pages) pg = 0;            // (flagged where the tiles were read)
    const size_t blk = (size_t)pg * a.pv.H + h;
    const size_t c0 = ((blk << a.pv.p_shift) + (k & (a.pv.P - 1))) * D + lane * V;
    const float sk = a.pv.k_scale[blk], sv = a.pv.v_scale[blk];
    float kc[V], vc[V], s = 0.0f;
#pragma unroll
    for (int p = 0; p < V / 2; ++p) {
      const uint32_t kw = cvt_e4m3x2_to_f16x2(reinterpret_cast<const uint16_t*>(a.pv.k_codes + c0)[p]);
      const uint32_t vw = cvt_e4m3x2_to_f16x2(reinterpret_cast<const uint16_t*>(a.pv.v_codes + c0)[p]);
      const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kw));
      const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&vw));
      kc[2 * p] = kf.x * sk;                             // the key's own size: queries may be as large as it is small
      kc[2 * p + 1] = kf.y * sk;
      vc[2 * p] = vf.x;
      vc[2 * p + 1] = vf.y;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) s = fmaf(x[c], kc[c], s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    const float y = s * a.scale_log2;
    const float mn = fmaxf(m, y);
    const float al = mn > m ? ex2f(m - mn) : 1.0f, w = y == -INFINITY ? 0.0f : ex2f(y - mn);
    m = mn;
    l = l * al + w;
#pragma unroll
    for (int c = 0; c < V; ++c) o[c] = o[c] * al + w * vc[c] * sv;
  }
  if (dst) {
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int p = 0; p < V / 2; ++p)
      reinterpret_cast<uint32_t*>(dst + lane * V)[p] = pack2<T>(o[2 * p] * inv, o[2 * p + 1] * inv);
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) o_at[lane * V + c] = o[c];
    if (lane == 0) *ml = make_float2(m + head, l);
  }
}

}  // namespace kvring_dev
