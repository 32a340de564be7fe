// paged_append: new keys and values into the pages of a paged FP8 cache.
//
// For each (page touched, key head, K or V): the new rows are read once, K is
// rotated (fp32, the ring write's operations), their absolute maximum a gives
// the block scale s = 2^k, the smallest power of two with a <= 448 s; a page
// that already held rows keeps its scale unless s is larger, and then its
// older codes are rounded again at the larger scale.  Both steps of the scale
// are powers of two, so a code that stays normal is carried over exactly:
// what a page holds does not depend on how many calls filled it, but for
// codes that become e4m3 subnormals (half a step of 2^-10 s).  That is why
// the scale is not a / 448, which would round every older code at each growth.
#include "paged.h"
#include "launch.h"

namespace kvring_dev {

// Block = 128 threads on one (page task, key head, K or V).  A row is handled
// by L = D / 16 lanes of 16 channels each, ROWS = 128 / L rows at a time, and
// a thread keeps the 16 fp32 values of up to P / ROWS rows until the block's
// maximum is known, so the input is read once.
//
// Tasks: sequence b touches at most floor(n_b / P) + 2 pages, so it owns the
// task numbers base(b) .. base(b + 1) - 1 with base(b) = floor(seq_start[b] /
// P) + 2 b; the block finds its b by counting the bases at or below its own
// number, all sequences in parallel.
template <int L, int P, typename T>
__global__ void __launch_bounds__(128) paged_append_kernel(PagedView pv, PagedBatch pb, const T* __restrict__ k,
                                                           long long k_stride, const T* __restrict__ v,
                                                           long long v_stride, const int32_t* __restrict__ pos) {
  constexpr int D = L * 16;
  constexpr int ROWS = 128 / L;                         // rows per pass
  constexpr int PASS = P > ROWS ? P / ROWS : 1;
  const int tid = threadIdx.x;
  // K and V of every head of a page are neighbouring blocks: together they
  // read whole input rows, and the same rows of the RoPE table
  const int task = blockIdx.x / (2 * pv.H);
  const int h = (blockIdx.x - task * 2 * pv.H) >> 1;
  const bool is_v = blockIdx.x & 1;
  pdl_wait();
  pdl_trigger();
  int b = -1;
  for (int i0 = 0; i0 < pb.n_seqs; i0 += 128) {
    const int i = i0 + tid;
    const bool below = i < pb.n_seqs && (min(max(__ldg(pb.seq_start + i), 0), pb.n_tokens) >> pv.p_shift) + 2 * i <= task;
    b += __syncthreads_count(below);
  }
  if (b < 0) return;
  bool ok;
  const SeqInfo s = seq_info(pb, pv.p_shift, b, ok);
  ok = ok && s.n <= s.len;
  const int j = ok ? task - ((s.s0 >> pv.p_shift) + 2 * b) : 0;
  if (!ok) {
    if (tid == 0) atomicOr(&pv.state[PST_ERR], DEVERR_SEQ);
    return;
  }
  const int first = s.len - s.n;                        // cache index of the first new token
  const int slot = (first >> pv.p_shift) + j;           // the task's page of the sequence
  const int lo = max(first, slot << pv.p_shift);
  const int hi = min(s.len, (slot + 1) << pv.p_shift);
  if (j < 0 || lo >= hi) return;
  const int page = __ldg(pb.table + b * pb.table_stride + slot);
  if (page < 0 || page >= pv.n_pages) {
    if (tid == 0) atomicOr(&pv.state[PST_ERR], DEVERR_PAGE);
    return;
  }
  const int held = lo - (slot << pv.p_shift);           // rows of the page that were there before
  const int cnt = hi - lo;
  const int tok0 = s.s0 + (lo - first);
  const int lane = tid % L;
  const int row = tid / L;
  const size_t blk = (size_t)page * pv.H + h;
  uint8_t* codes = (is_v ? pv.v_codes : pv.k_codes) + blk * (size_t)(P * D) + lane * 16;
  float* scale_at = (is_v ? pv.v_scale : pv.k_scale) + blk;
  const float old = held > 0 ? *scale_at : 0.0f;

  float x[PASS][16];
  float amax = 0.0f;
  bool bad = false;
  const RopeLane rl = rope_lane(pv, lane * 8);
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * ROWS + row;
    if (r < cnt) {
      const int tok = tok0 + r;
      const uint4* src = reinterpret_cast<const uint4*>((is_v ? v + tok * v_stride : k + tok * k_stride) +
                                                        (size_t)h * D + lane * 16);
      const uint4 a0 = __ldg(src), a1 = __ldg(src + 1);
      load8_f32<T>(a0, x[p]);
      load8_f32<T>(a1, x[p] + 8);
      if (!is_v) {
        float2 cs[8];
        rope_load(pv, rl, pos + (size_t)tok * pv.n_axes, cs, bad);
#pragma unroll
        for (int m = 0; m < 8; ++m) rope_pair(x[p][2 * m], x[p][2 * m + 1], cs[m].x, cs[m].y);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[p][i]));
    }
  }
  if (bad) atomicOr(&pv.state[PST_ERR], DEVERR_POS_RANGE);
  __shared__ float wmax[4];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  if ((tid & 31) == 0) wmax[tid >> 5] = amax;
  __syncthreads();                                      // also: every thread has read the old scale
  amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
  float scale, inv;
  pow2_scale(amax, scale, inv);
  if (scale <= old) {
    scale = old;
    inv = old > 0.0f ? 1.0f / old : 0.0f;               // a power of two: exact
  } else if (held > 0) {
    // the page's older codes at the larger scale (a row of zeros for old = 0)
    const float ratio = old * inv;
    for (int r = row; r < held; r += ROWS) {
      uint4* at = reinterpret_cast<uint4*>(codes + r * D);
      float y[16];
      dequant16_codes(*at, y);
      *at = quant16(y, ratio);
    }
  }
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * ROWS + row;
    if (r < cnt) *reinterpret_cast<uint4*>(codes + (held + r) * D) = quant16(x[p], inv);
  }
  if (tid == 0) *scale_at = scale;
}

// ---------------------------------------------------------------- RoPE table
// (cos, sin) of pos * omega_j, the angle and both functions in fp64, rounded
// once to fp32.
__global__ void __launch_bounds__(256) paged_rope_kernel(float2* table, int pos_min, int pos_count, int pairs,
                                                         const double* __restrict__ omega) {
  const long long n = (long long)pos_count * pairs;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int p = (int)(i / pairs);
    double s, c;
    sincos((double)(pos_min + p) * omega[(int)(i - (long long)p * pairs)], &s, &c);
    table[i] = make_float2((float)c, (float)s);
  }
}

cudaError_t launch_paged_rope_table(float2* table, int pos_min, int pos_count, int pairs, const double* omega,
                                    cudaStream_t st) {
  const long long n = (long long)pos_count * pairs;
  const long long blocks = (n + 255) / 256;
  paged_rope_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(table, pos_min, pos_count, pairs, omega);
  return cudaGetLastError();
}

template <int L, int P, typename T>
static cudaError_t append_t(const PagedView& pv, const PagedBatch& pb, const void* k, long long k_stride,
                            const void* v, long long v_stride, const int32_t* pos, cudaStream_t st) {
  const dim3 grid((unsigned)((pb.n_tokens / P + 2 * pb.n_seqs) * 2 * pv.H));
  return launch_pdl(paged_append_kernel<L, P, T>, grid, dim3(128), 0, st, pv, pb, static_cast<const T*>(k), k_stride,
                    static_cast<const T*>(v), v_stride, pos);
}

template <int L, typename T>
static cudaError_t append_p(const PagedView& pv, const PagedBatch& pb, const void* k, long long k_stride,
                            const void* v, long long v_stride, const int32_t* pos, cudaStream_t st) {
  switch (pv.P) {
    case 16: return append_t<L, 16, T>(pv, pb, k, k_stride, v, v_stride, pos, st);
    case 32: return append_t<L, 32, T>(pv, pb, k, k_stride, v, v_stride, pos, st);
    case 64: return append_t<L, 64, T>(pv, pb, k, k_stride, v, v_stride, pos, st);
    default: return append_t<L, 128, T>(pv, pb, k, k_stride, v, v_stride, pos, st);
  }
}

cudaError_t launch_paged_append(const PagedView& pv, const PagedBatch& pb, const void* k, long long k_stride,
                                const void* v, long long v_stride, const int32_t* pos, bool f16, cudaStream_t st) {
  if (pv.D == 64)
    return f16 ? append_p<4, __half>(pv, pb, k, k_stride, v, v_stride, pos, st)
               : append_p<4, __nv_bfloat16>(pv, pb, k, k_stride, v, v_stride, pos, st);
  return f16 ? append_p<8, __half>(pv, pb, k, k_stride, v, v_stride, pos, st)
             : append_p<8, __nv_bfloat16>(pv, pb, k, k_stride, v, v_stride, pos, st);
}

}  // namespace kvring_dev
