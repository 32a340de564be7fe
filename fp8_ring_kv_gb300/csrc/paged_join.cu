// paged_join: the items of the paged attention that several workers (warps of
// the row kernel, blocks of the tile kernel) share.
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
#pragma unroll 8
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
    l = l * f0 + (some ? ml.y * f1 : ml.y);              // no key: 0; scores all NaN: NaN
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = some ? o[i] * f0 + x[i] * f1 : o[i];
  }
}

// Block x looks at the records of ``per`` workers (at most 32, a lane each).
// Few rows per item (TR <= 16): of an item of few pieces, row y to the warp
// that has the record; of one of many pieces (a long sequence spread over the
// GPU), row y to the whole block, warp i the pieces i, i + JW, ...
// Many rows (one record per block): a row to a warp.
constexpr int JW = 8;                                    // warps
template <int D, int TR, typename T>
__device__ __forceinline__ void join_items(const PagedAttn& a, const PieceScratch& ps, int workers, int per,
                                           float (&acc)[JW][D], float2 (&mls)[JW]) {
  constexpr int V = D / 32;                              // channels per lane
  // pieces from which a whole block joins a row (one context of 300 tokens: 12.7 us
  // against 13.7 with 12; two of 130,000: 90.4 against 108.7 with one warp for all)
  constexpr int MANY = 4;
  constexpr bool TALL = TR > 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w0 = blockIdx.x * per;
  PieceRec mine = {};
  if (lane < per && w0 + lane < workers) mine = ps.rec[w0 + lane];
  const bool long_ = !TALL && mine.last - (w0 + lane) >= MANY;
  unsigned few = __ballot_sync(0xFFFFFFFFu, mine.rows > 0 && !long_);
  unsigned many = __ballot_sync(0xFFFFFFFFu, mine.rows > 0 && long_);
  auto record = [&](int i) {
    PieceRec r;
    r.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, i);
    r.last = __shfl_sync(0xFFFFFFFFu, mine.last, i);
    r.h = __shfl_sync(0xFFFFFFFFu, mine.h, i);
    r.s0 = __shfl_sync(0xFFFFFFFFu, mine.s0, i);
    r.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, i);
    return r;
  };
  auto out_row = [&](const PieceRec& it, int r) {
    const int rr = it.row0 + r;
    const int i = rr / a.pv.G;
    return reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + (it.s0 + i) * a.out_stride +
                                       (size_t)(it.h * a.pv.G + rr - i * a.pv.G) * D);
  };
  float m, l, o[V];
  for (int k = 0; few; ++k, few &= few - 1) {
    const int i = __ffs(few) - 1;
    if (!TALL && k % JW != warp) continue;
    const PieceRec it = record(i);
    for (int r = TALL ? blockIdx.y * JW + warp : blockIdx.y; r < it.rows; r += gridDim.y * (TALL ? JW : 1)) {
      sum_pieces<V, TR>(ps, w0 + i, w0 + i, 1, it.last, r, m, l, o);
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      uint32_t* dst = out_row(it, r) + lane * (V / 2);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) dst[c] = pack2<T>(o[2 * c] * inv, o[2 * c + 1] * inv);
    }
  }
  for (; many; many &= many - 1) {                       // the same in every warp
    const int i = __ffs(many) - 1;
    const PieceRec it = record(i);
    for (int r = blockIdx.y; r < it.rows; r += gridDim.y) {
      sum_pieces<V, TR>(ps, w0 + i, w0 + i + warp, JW, it.last, r, m, l, o);
      if (lane == 0) mls[warp] = make_float2(m, l);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[warp][lane * V + c] = o[c];
      __syncthreads();
      if (tid < D / 2) {
        float mm = -INFINITY, ll = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
        for (int k = 0; k < JW; ++k) mm = fmaxf(mm, mls[k].x);
#pragma unroll
        for (int k = 0; k < JW; ++k) {
          const float f = mls[k].x != -INFINITY ? ex2f(mls[k].x - mm) : 1.0f;   // no key: zeros
          ll += mls[k].y * f;
          o0 += acc[k][2 * tid] * f;
          o1 += acc[k][2 * tid + 1] * f;
        }
        const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
        out_row(it, r)[tid] = pack2<T>(o0 * inv, o1 * inv);
      }
      __syncthreads();
    }
  }
}

// The row kernel's items and, blockIdx.z = 1, the tile kernel's.
constexpr int JOIN_RECORDS = 8;                          // of the row kernel's, per block
template <int D, typename T>
__global__ void __launch_bounds__(32 * JW) paged_join_kernel(const __grid_constant__ PagedAttn a, int workers, int blocks) {
  __shared__ float acc[JW][D];
  __shared__ float2 mls[JW];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.z == 0) join_items<D, kRowsTile<T>, T>(a, a.rows, workers, JOIN_RECORDS, acc, mls);
  else join_items<D, kTilesRows, T>(a, a.tiles, blocks, 1, acc, mls);
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
static cudaError_t join_t(const PagedAttn& a, bool tiles, int blocks, cudaStream_t st) {
  const long long most = (long long)a.max_new * a.pv.G;
  const int workers = blocks * paged_rows_warps(a, std::is_same_v<T, __half>);
  const int x = (workers + JOIN_RECORDS - 1) / JOIN_RECORDS;
  static_assert(kTilesRows % (4 * JW) == 0);
  const dim3 grid = tiles ? dim3(x > blocks ? x : blocks, kTilesRows / JW / 4, 2)
                          : dim3(x, (unsigned)(most < kRowsTile<T> ? most : kRowsTile<T>));
  return launch_pdl(paged_join_kernel<D, T>, grid, dim3(32 * JW), 0, st, a, workers, blocks);
}

static cudaError_t launch_paged_join(const PagedAttn& a, bool tiles, bool f16, int blocks, cudaStream_t st) {
  if (a.pv.D == 64)
    return f16 ? join_t<64, __half>(a, tiles, blocks, st) : join_t<64, __nv_bfloat16>(a, tiles, blocks, st);
  return f16 ? join_t<128, __half>(a, tiles, blocks, st) : join_t<128, __nv_bfloat16>(a, tiles, blocks, st);
}

// ---------------------------------------------------------------- one call
// The kernel of few rows always runs (only the device knows how many new
// tokens each sequence has), the kernel of many where max_new allows such.
cudaError_t launch_paged_attend(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int sms,
                                cudaStream_t st) {
  const int blocks = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  const bool many = (long long)a.max_new * a.pv.G > kRowsMax;
  cudaError_t e = launch_paged_rows(a, tmK, tmV, f16, blocks, st);
  if (e == cudaSuccess && many) e = launch_paged_tiles(a, tmK, tmV, f16, blocks, st);
  return e == cudaSuccess ? launch_paged_join(a, many, f16, blocks, st) : e;
}

}  // namespace kvring_dev
