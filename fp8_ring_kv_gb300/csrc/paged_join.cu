// paged_join: the items of the paged attention that several workers share.
//
//   out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i
// over the pieces in the workers' order (no atomics: the result does not
// depend on which worker came first).
#include "paged.h"
#include "launch.h"

namespace kvring_dev {

// The sum over pieces p, p + step, ... <= last of one row: lane i holds
// channels V i .. V i + V - 1.  Worker w's own piece is slot 2 w + 1, the
// pieces of the workers after it slots 2 p.
template <int V, int TR>
__device__ __forceinline__ void sum_pieces(const PieceScratch& ps, int w, int p, int step, int last, int r, float& m,
                                           float& l, float (&o)[V]) {
  constexpr int D = 32 * V;
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
#pragma unroll 4
  for (; p <= last; p += step) {
    const size_t row = (size_t)(2 * p + (p == w ? 1 : 0)) * TR + r;
    const float2 ml = ps.ml[row];
    float x[V];
    if constexpr (V == 4) {
      const float4 f = reinterpret_cast<const float4*>(ps.o + row * D)[lane];
      x[0] = f.x;
      x[1] = f.y;
      x[2] = f.z;
      x[3] = f.w;
    } else {
      const float2 f = reinterpret_cast<const float2*>(ps.o + row * D)[lane];
      x[0] = f.x;
      x[1] = f.y;
    }
    const bool some = ml.x != -INFINITY;                 // else x was not written
    const float mn = some ? fmaxf(m, ml.x) : m;
    const float f0 = mn > m ? ex2f(m - mn) : 1.0f, f1 = some ? ex2f(ml.x - mn) : 0.0f;
    m = mn;
    l = l * f0 + (some ? ml.y * f1 : 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = some ? o[i] * f0 + x[i] * f1 : o[i];
  }
}

// Block x looks at the records of workers 8 x .. 8 x + 7 (TR <= 16) or at that
// of worker x, and takes rows y, y + gridDim.y, ... of its items.  An item of
// few pieces: a row to a warp (a record to a warp, or the rows shared by the
// warps); one of many (a long sequence spread over the GPU): a row to all eight
// warps, warp i the pieces i, i + 8, ...
template <int D, int TR, typename T>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedAttn a, PieceScratch ps,
                                                         int workers) {
  constexpr int RECS = TR <= 16 ? 8 : 1;
  constexpr int V = D / 32;                              // channels per lane
  constexpr int MANY = 12;                               // pieces
  __shared__ float acc[8][D];
  __shared__ float2 mls[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  struct Item {
    PieceRec rec;
    int w, rows, s0;
  };
  auto item = [&](int w) {
    Item it;
    it.w = w;
    it.rec.b = -1;
    if (w < workers) it.rec = ps.rec[w];
    it.rows = 0;
    if (it.rec.b >= 0) {
      bool ok;
      const SeqInfo s = seq_info(a.pb, a.pv.p_shift, it.rec.b, ok);
      it.rows = min(s.n * a.pv.G - it.rec.tile * TR, TR);
      it.s0 = s.s0;
    }
    return it;
  };
  auto out_row = [&](const Item& it, int r) {
    const int rr = it.rec.tile * TR + r;
    const int i = rr / a.pv.G;
    return static_cast<T*>(a.out) + (it.s0 + i) * a.out_stride + (size_t)(it.rec.h * a.pv.G + rr - i * a.pv.G) * D;
  };
  float m, l, o[V];
  bool many;
  {
    const Item it = item(RECS == 8 ? blockIdx.x * 8 + warp : blockIdx.x);
    many = it.rec.b >= 0 && it.rec.last - it.w >= MANY;
    if (!many)
      for (int r = RECS == 8 ? blockIdx.y : blockIdx.y * 8 + warp; r < it.rows; r += gridDim.y * (RECS == 8 ? 1 : 8)) {
        sum_pieces<V, TR>(ps, it.w, it.w, 1, it.rec.last, r, m, l, o);
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        uint32_t* dst = reinterpret_cast<uint32_t*>(out_row(it, r)) + lane * (V / 2);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dst[i] = pack2<T>(o[2 * i] * inv, o[2 * i + 1] * inv);
      }
  }
  if (!__syncthreads_or(many)) return;
  for (int w0 = 0; w0 < RECS; ++w0) {
    const Item it = item(blockIdx.x * RECS + w0);
    if (it.rec.b < 0 || it.rec.last - it.w < MANY) continue;
    for (int r = blockIdx.y; r < it.rows; r += gridDim.y) {
      sum_pieces<V, TR>(ps, it.w, it.w + warp, 8, it.rec.last, r, m, l, o);
      if (lane == 0) mls[warp] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[warp][lane * V + i] = o[i];
      __syncthreads();
      if (tid < D / 2) {
        float mm = -INFINITY, ll = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mm = fmaxf(mm, mls[i].x);
        if (mm != -INFINITY) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float f = ex2f(mls[i].x - mm);
            ll += mls[i].y * f;
            o0 += acc[i][2 * tid] * f;
            o1 += acc[i][2 * tid + 1] * f;
          }
        }
        const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
        reinterpret_cast<uint32_t*>(out_row(it, r))[tid] = pack2<T>(o0 * inv, o1 * inv);
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- scratch
static size_t piece_bytes(int workers, int rows, int D) {
  const size_t slots = (size_t)2 * workers * rows;
  return slots * D * 4 + slots * 8 + (size_t)workers * sizeof(PieceRec);
}

static uint8_t* carve(uint8_t* at, int workers, int rows, int D, PieceScratch* ps) {
  const size_t slots = (size_t)2 * workers * rows;
  ps->o = reinterpret_cast<float*>(at);
  ps->ml = reinterpret_cast<float2*>(at + slots * D * 4);
  ps->rec = reinterpret_cast<PieceRec*>(at + slots * D * 4 + slots * 8);
  return at + piece_bytes(workers, rows, D);
}

size_t paged_scratch_bytes(int D) {
  return piece_bytes(kRowsWorkersMax, 16, D) + piece_bytes(kPagedMaxSms, kTilesRows, D);
}

void paged_carve_scratch(uint8_t* base, int D, PagedAttn* a) {
  carve(carve(base, kRowsWorkersMax, 16, D, &a->rows), kPagedMaxSms, kTilesRows, D, &a->tiles);
}

template <int D, typename T>
static cudaError_t join_t(const PagedAttn& a, bool tiles, int workers, cudaStream_t st) {
  if (tiles)
    return launch_pdl(paged_join_kernel<D, kTilesRows, T>, dim3(workers, 8), dim3(256), 0, st, a, a.tiles, workers);
  const long long most = (long long)a.max_new * a.pv.G;
  const unsigned rows = (unsigned)(most < kRowsMax<T> ? most : kRowsMax<T>);
  return launch_pdl(paged_join_kernel<D, kRowsMax<T>, T>, dim3((workers + 7) / 8, rows), dim3(256), 0, st, a, a.rows,
                    workers);
}

cudaError_t launch_paged_join(const PagedAttn& a, bool tiles, bool f16, int workers, cudaStream_t st) {
  if (a.pv.D == 64)
    return f16 ? join_t<64, __half>(a, tiles, workers, st) : join_t<64, __nv_bfloat16>(a, tiles, workers, st);
  return f16 ? join_t<128, __half>(a, tiles, workers, st) : join_t<128, __nv_bfloat16>(a, tiles, workers, st);
}

// ---------------------------------------------------------------- one call
cudaError_t launch_paged_attend(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int sms,
                                cudaStream_t st) {
  const int blocks = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  const int few = f16 ? kRowsMax<__half> : kRowsMax<__nv_bfloat16>;
  const bool many = (long long)a.max_new * a.pv.G > few;
  cudaError_t e = launch_paged_rows(a, tmK, tmV, f16, blocks, st);
  if (e == cudaSuccess && many) e = launch_paged_tiles(a, tmK, tmV, f16, blocks, st);
  if (e == cudaSuccess) e = launch_paged_join(a, false, f16, blocks * paged_rows_warps(a, f16), st);
  if (e == cudaSuccess && many) e = launch_paged_join(a, true, f16, blocks, st);
  return e;
}

}  // namespace kvring_dev
