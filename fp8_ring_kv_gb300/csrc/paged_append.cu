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
//
// What bounds it: a thread's chain of dependent loads (the sequences' numbers,
// positions, table rows) with as many threads on an SM as the registers of two
// rows each allow.  16,662 tokens of 8 heads x 128: 26.5 us, 3.9 TB/s of the
// input's and codes' bytes, 57% of a copy (without the bound on registers
// 31 us; several units per block one after the other 39 us, the loop's registers
// spilt).
#include "paged.h"
#include "launch.h"

namespace kvring_dev {

// Tokens per sequence, on average, up to which the kernel of few tokens is
// taken.  128 sequences, 8 heads x 128, pages of 64, in us, against whole pages:
// 1 token each 3.2 : 10.7, 4 tokens 6.0 : 10.9, 16 tokens 16.2 : 11.7, 64 tokens
// 41 : 21; 16 sequences of 256 tokens 52 : 9.  Well below the crossing, because
// the average may hide one long sequence.
constexpr int kAppendFew = 4;

// Tasks: sequence b touches at most floor(n_b / P) + 2 pages, so it owns the
// task numbers base(b) .. base(b + 1) - 1 with base(b) = floor(seq_start[b] /
// P) + 2 b; a block looks for the sequence that owns its number, all sequences
// in parallel.  (Sequences whose numbers hold own separate tasks, however wrong
// those of others are, unless starts that decrease make them overlap.)
struct AppendTask {
  int held;       // rows of the page that were there before
  int cnt;        // new rows
  int tok0;       // the first one's token
  int page;       // -1: nothing to do
};

// ``found``: one word of shared memory, -1 at first.
__device__ AppendTask append_task(const PagedView& pv, const PagedBatch& pb, int task, int* found) {
  const int tid = threadIdx.x;
  AppendTask t = {0, 0, 0, -1};
  for (int i = tid; i < pb.n_seqs; i += blockDim.x) {
    bool ok;
    const SeqInfo s = seq_info(pb, pv.p_shift, i, ok);
    ok = ok && s.n <= s.len;
    if (!ok && blockIdx.x == 0) atomicOr(&pv.state[PST_ERR], DEVERR_SEQ);
    const int j = task - (s.s0 >> pv.p_shift) - 2 * i;
    const int first = s.len - s.n;
    if (ok && s.n > 0 && j >= 0 && j <= ((s.len - 1) >> pv.p_shift) - (first >> pv.p_shift)) atomicMax(found, i);
  }
  __syncthreads();
  const int b = *found;
  if (b < 0) return t;
  const int s0 = pb.seq_start[b], s1 = pb.seq_start[b + 1], len = pb.kv_len[b];
  const int j = task - (s0 >> pv.p_shift) - 2 * b;
  const int first = len - (s1 - s0);                    // cache index of the first new token
  const int slot = (first >> pv.p_shift) + j;           // the task's page of the sequence
  const int lo = max(first, slot << pv.p_shift);
  const int hi = min(len, (slot + 1) << pv.p_shift);
  t.held = lo - (slot << pv.p_shift);
  t.cnt = hi - lo;
  t.tok0 = s0 + (lo - first);
  t.page = pb.table[b * pb.table_stride + slot];
  if (t.page < 0 || t.page >= pv.n_pages) {
    if (tid == 0) atomicOr(&pv.state[PST_ERR], DEVERR_PAGE);
    t.page = -1;
  }
  return t;
}

// Codes of x * inv in a block of scale 2^k, or (zero) in one of scale 0: +0
// there, but for a NaN, which is 0x7F in any block.
__device__ __forceinline__ uint4 block_codes(const float* x, float inv, bool zero) {
  if (!zero) return codes16(x, inv);
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i] != x[i] ? x[i] : 0.0f;
  return codes16(y, 1.0f);
}

// The scale that a block of codes takes, and its inverse; true where it grew.
__device__ __forceinline__ bool block_scale(float amax, float old, float& scale, float& inv) {
  pow2_scale(amax, scale, inv);
  if (scale > old) return true;
  scale = old;
  inv = old > 0.0f ? 1.0f / old : 0.0f;                 // a power of two: exact
  return false;
}

// Whole pages: a block on one unit (page task, key head, K or V).  A row is
// handled by L = D / 16 lanes of 16 channels each; a thread keeps the fp32
// values of two rows until the block's maximum is known, so the input is read
// once.  More rows per thread would take the registers of the warps that hide
// the loads' latency, fewer make blocks whose barrier waits for more warps
// (pages of 64 x 128: one row 41 us against 26.5, four rows 28; pages of 16 x 64,
// 20,540 tokens of 24 heads: blocks of 128 threads 134 us, of 32 threads 66).
// K and V of every head of a page are neighbouring blocks: together they read
// whole input rows, and the same rows of the RoPE table.
template <int L, int P>
constexpr int append_threads = P * L / 2;

template <int L, int P, typename T>
__global__ void __launch_bounds__(append_threads<L, P>, 1024 / append_threads<L, P>)
    paged_append_kernel(PagedView pv, PagedBatch pb, const T* k, long long k_stride,
                        const T* v, long long v_stride, const int32_t* pos) {
  constexpr int D = L * 16;
  constexpr int THREADS = append_threads<L, P>;
  constexpr int ROWS = THREADS / L;                     // rows per pass
  constexpr int PASS = 2;
  static_assert(THREADS % 32 == 0 && ROWS * PASS == P);
  __shared__ int found;
  __shared__ float wmax[THREADS / 32];
  const int tid = threadIdx.x;
  const int task = blockIdx.x / (2 * pv.H);
  const int h = (blockIdx.x - task * 2 * pv.H) >> 1;
  const bool is_v = blockIdx.x & 1;
  if (tid == 0) found = -1;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const AppendTask t = append_task(pv, pb, task, &found);
  if (t.cnt == 0) return;                               // the whole block
  const int lane = tid % L;
  const int row = tid / L;
  const T* src0 = (is_v ? v + t.tok0 * v_stride : k + t.tok0 * k_stride) + (size_t)h * D + lane * 16;
  const long long stride = is_v ? v_stride : k_stride;
  float x[PASS][16];
  float amax = 0.0f;
  bool bad = false;
  const RopeLane rl = rope_lane(pv, lane * 8);
  uint4 raw[PASS][2];
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * ROWS + row;
    raw[p][0] = raw[p][1] = make_uint4(0, 0, 0, 0);
    if (r < t.cnt) {
      const uint4* src = reinterpret_cast<const uint4*>(src0 + r * stride);
      raw[p][0] = src[0];
      raw[p][1] = src[1];
    }
  }
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * ROWS + row;
    load8_f32<T>(raw[p][0], x[p]);
    load8_f32<T>(raw[p][1], x[p] + 8);
    if (!is_v && r < t.cnt) {
      float2 cs[8];
      rope_load(pv, rl, pos + (size_t)(t.tok0 + r) * pv.n_axes, cs, bad);
#pragma unroll
      for (int m = 0; m < 8; ++m) rope_pair(x[p][2 * m], x[p][2 * m + 1], cs[m].x, cs[m].y);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[p][i]));
  }
  if (bad) atomicOr(&pv.state[PST_ERR], DEVERR_POS_RANGE);
  if (t.page < 0) return;                               // the whole block
  const size_t blk = (size_t)t.page * pv.H + h;
  uint8_t* codes = (is_v ? pv.v_codes : pv.k_codes) + blk * (size_t)(P * D) + lane * 16;
  float* scale_at = (is_v ? pv.v_scale : pv.k_scale) + blk;
  const float old = t.held > 0 ? *scale_at : 0.0f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
  if ((tid & 31) == 0) wmax[tid >> 5] = amax;
  __syncthreads();                                      // also: every thread has read the old scale
  amax = wmax[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) amax = fmaxf(amax, wmax[i]);
  float scale, inv;
  if (block_scale(amax, old, scale, inv) && t.held > 0) {
    // the page's older codes at the larger scale (zeros and NaN for old = 0)
    const float ratio = old * inv;
    for (int r = row; r < t.held; r += ROWS) {
      uint4* at = reinterpret_cast<uint4*>(codes + r * D);
      float y[16];
      dequant16_codes(*at, y);
      *at = block_codes(y, ratio, old == 0.0f);
    }
  }
#pragma unroll
  for (int p = 0; p < PASS; ++p) {
    const int r = p * ROWS + row;
    if (r < t.cnt) *reinterpret_cast<uint4*>(codes + (t.held + r) * D) = block_codes(x[p], inv, scale == 0.0f);
  }
  if (tid == 0) *scale_at = scale;
}

// A few tokens per sequence (decoding): a block on one page task, L lanes on
// each (key head, K or V) of it, its rows one after the other: the lanes of a
// row are all that its maximum needs, so nothing waits for a barrier, and a
// token's heads are one block instead of 2 H.  Right for any number of rows (it
// reads them twice), slow for many.
template <int L, typename T>
__global__ void __launch_bounds__(512)
    paged_append_few_kernel(PagedView pv, PagedBatch pb, const T* k, long long k_stride,
                            const T* v, long long v_stride, const int32_t* pos) {
  constexpr int D = L * 16;
  __shared__ int found;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const AppendTask t = append_task(pv, pb, blockIdx.x, &found);
  if (t.cnt == 0) return;
  const int lane = threadIdx.x % L;
  const unsigned group = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
  const RopeLane rl = rope_lane(pv, lane * 8);
  bool bad = false;
  for (int unit = threadIdx.x / L; unit < 2 * pv.H; unit += blockDim.x / L) {
    const int h = unit >> 1;
    const bool is_v = unit & 1;
    const T* src0 = (is_v ? v + t.tok0 * v_stride : k + t.tok0 * k_stride) + (size_t)h * D + lane * 16;
    const long long stride = is_v ? v_stride : k_stride;
    auto load = [&](int r, float (&x)[16]) {
      const uint4* src = reinterpret_cast<const uint4*>(src0 + r * stride);
      const uint4 a0 = src[0], a1 = src[1];
      float2 cs[8];
      if (!is_v) rope_load(pv, rl, pos + (size_t)(t.tok0 + r) * pv.n_axes, cs, bad);
      load8_f32<T>(a0, x);
      load8_f32<T>(a1, x + 8);
      if (!is_v) {
#pragma unroll
        for (int m = 0; m < 8; ++m) rope_pair(x[2 * m], x[2 * m + 1], cs[m].x, cs[m].y);
      }
    };
    float x[16];
    float amax = 0.0f;
#pragma unroll 2
    for (int r = t.cnt - 1; r >= 0; --r) {              // ends with row 0's values in x
      load(r, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
    }
    if (t.page < 0) continue;
    const size_t blk = (size_t)t.page * pv.H + h;
    uint8_t* codes = (is_v ? pv.v_codes : pv.k_codes) + (blk << pv.p_shift) * D + lane * 16;
    float* scale_at = (is_v ? pv.v_scale : pv.k_scale) + blk;
    const float old = t.held > 0 ? *scale_at : 0.0f;
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, off));
    float scale, inv;
    if (block_scale(amax, old, scale, inv) && t.held > 0) {
      const float ratio = old * inv;
      for (int r = 0; r < t.held; ++r) {
        uint4* at = reinterpret_cast<uint4*>(codes + r * D);
        float y[16];
        dequant16_codes(*at, y);
        *at = block_codes(y, ratio, old == 0.0f);
      }
    }
#pragma unroll 2
    for (int r = 0; r < t.cnt; ++r) {
      if (r > 0) load(r, x);
      *reinterpret_cast<uint4*>(codes + (t.held + r) * D) = block_codes(x, inv, scale == 0.0f);
    }
    __syncwarp(group);                                  // every lane has read the old scale
    if (lane == 0) *scale_at = scale;
  }
  if (bad) atomicOr(&pv.state[PST_ERR], DEVERR_POS_RANGE);
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
    sincos(((double)pos_min + p) * omega[(int)(i - (long long)p * pairs)], &s, &c);
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
  const long long tasks = pb.n_tokens / P + 2 * pb.n_seqs;
  const T* kt = static_cast<const T*>(k);
  const T* vt = static_cast<const T*>(v);
  if (pb.n_tokens <= kAppendFew * pb.n_seqs) {
    const int units = 2 * pv.H * L;                     // threads that a token's heads keep busy
    const int threads = units < 128 ? 128 : units > 512 ? 512 : (units + 31) / 32 * 32;
    return launch_pdl(paged_append_few_kernel<L, T>, dim3((unsigned)tasks), dim3(threads), 0, st, pv, pb, kt, k_stride,
                      vt, v_stride, pos);
  }
  return launch_pdl(paged_append_kernel<L, P, T>, dim3((unsigned)(tasks * 2 * pv.H)), dim3(append_threads<L, P>), 0,
                    st, pv, pb, kt, k_stride, vt, v_stride, pos);
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
