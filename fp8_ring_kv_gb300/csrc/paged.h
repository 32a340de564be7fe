// Internal definitions of the paged FP8 KV cache: device views, the batch of
// sequences a call works on, and the kernels' host-side entry points.
#pragma once
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace kvring_dev {

// state words at the start of the workspace
enum : int { PST_ERR = 0, PST_WORDS = 64 };
// device error bits (beside DEVERR_POS_RANGE and DEVERR_TIMEOUT)
enum : int { DEVERR_SEQ = 8, DEVERR_PAGE = 16 };

constexpr int kPagedMaxSeqs = 2048;
constexpr int kPagedMaxLen = 1 << 22;    // tokens of one sequence
constexpr int kPagedMaxSms = 160;        // sizes the attention's scratch

// Device view of one layer of the cache, passed by value to the kernels.
struct PagedView {
  int32_t* state;                 // PST_* words
  const float2* rope[kMaxAxes];   // per axis: [pos_count][axis_dims/2] (cos, sin)
  int32_t pos_min[kMaxAxes];
  int32_t pos_count[kMaxAxes];
  int32_t axis_pairs[kMaxAxes];
  int32_t pair_off[kMaxAxes];
  uint8_t* k_codes;               // [n_pages][H][P][D]
  uint8_t* v_codes;
  float* k_scale;                 // [n_pages][H]
  float* v_scale;
  int32_t H, QH, G, D, P, p_shift, n_pages, n_axes;   // G = QH / H query heads per key head
  long long row0;                 // the layer's first row of the code arrays seen as rows of D
};

// The sequences of one call: sequence b's new tokens are rows seq_start[b] ..
// seq_start[b+1]-1 of the packed inputs, kv_len[b] its tokens in the cache
// once they are in, table[b * table_stride + j] its page j.
struct PagedBatch {
  const int32_t* seq_start;
  const int32_t* kv_len;
  const int32_t* table;
  long long table_stride;
  int32_t n_seqs, n_tokens, table_width;
};

// ---------------------------------------------------------------- attention work
// Rows of queries: sequence b has n_b * G rows per key head (row r: token
// r / G, query head h * G + r % G).  Two kernels share the sequences: those
// of at most kRowsMax rows go to the register-tile kernel (kRowsTile rows of
// one sequence and key head per item), the others to the tensor-memory kernel
// (256 rows per item).  fp16 queries take two of the register tile's 16 columns
// each (high and low part).
constexpr int kRowsWarps = 12, kRowsKeys = 32;   // warps of a block, at most; keys of a tile
template <typename T>
constexpr int kRowsTile = std::is_same_v<T, __half> ? 8 : 16;
// A batch of 16 contexts of 4,000 with 8 query heads per key head, in us, the
// register tiles against the tensor memory: 3 new tokens (24 rows) bf16 73
// against 78, fp16 79 against 106; 4 (32 rows) 76 against 78, 100 against 106;
// 5 (40 rows) 95 against 78.  64 contexts of 500, 4 tokens: 49 against 76.
constexpr int kRowsMax = 32;
constexpr int kTilesRows = 256;
constexpr int kRowsWorkersMax = kPagedMaxSms * kRowsWarps;

// What a worker leaves for the merge when an item it began ends in a later
// worker's range: the item, and the last worker that holds a piece of it.
struct alignas(16) PieceRec {
  int32_t rows;                   // of the item; 0: nothing to merge
  int32_t last, h, s0, row0;      // row0: its first row among the sequence's
  int32_t pad[3];
};

// Partial results: slot 2w holds the piece of an item begun before worker w's
// range, slot 2w + 1 the piece of an item that w began and did not end.
// o [slot][rows][D] fp32 (unnormalised), ml [slot][rows] (a reference in log2
// units, near the running maximum, and the sum); m = -inf marks rows (or whole
// pieces) without a key.
struct PieceScratch {
  float* o;
  float2* ml;
  PieceRec* rec;
};

struct PagedAttn {
  PagedView pv;
  PagedBatch pb;
  const void* q;
  const int32_t* q_pos;
  void* out;
  long long q_stride, out_stride;   // elements between tokens
  float scale_log2;                 // softmax scale * log2(e)
  int32_t causal, window, max_new;
  PieceScratch rows, tiles;
};

// bytes of the attention's scratch (the same on every device)
size_t paged_scratch_bytes(int D);
void paged_carve_scratch(uint8_t* base, int D, PagedAttn* a);

cudaError_t launch_paged_rope_table(float2* table, int pos_min, int pos_count, int pairs, const double* omega,
                                    cudaStream_t st);
cudaError_t launch_paged_append(const PagedView& pv, const PagedBatch& pb, const void* k, long long k_stride,
                                const void* v, long long v_stride, const int32_t* pos, bool f16, cudaStream_t st);
cudaError_t prepare_paged_rows(int D);
cudaError_t prepare_paged_tiles(int D);
// the kernel of few rows, and the kernel of many; ``blocks`` of either share its work
int paged_rows_warps(const PagedAttn& a, bool f16);   // workers per block of this call
cudaError_t launch_paged_rows(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                              cudaStream_t st);
cudaError_t launch_paged_tiles(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                               cudaStream_t st);
// tmK, tmV: the code arrays as [rows][D] u8, box {D, min(P, 32)}
cudaError_t launch_paged_attend(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int sms,
                                cudaStream_t st);

// ---------------------------------------------------------------- sequences
struct SeqInfo {
  int s0, n, len;
};

// What another kernel may have written just before (the batch's numbers and
// rows, codes and scales) is read with plain loads: a kernel launched ahead of
// that one's end (dependent launch) must not use the read-only path, which may
// answer with what the SM fetched before.  Only the RoPE tables never change.

// Sequence b's numbers.  Ones that contradict each other or the call's sizes
// give n = 0 (the sequence is left out) and ok = false.
__device__ __forceinline__ SeqInfo seq_info(const PagedBatch& pb, int p_shift, int b, bool& ok) {
  SeqInfo s;
  s.s0 = pb.seq_start[b];
  const int s1 = pb.seq_start[b + 1];
  s.len = pb.kv_len[b];
  ok = s.s0 >= 0 && s1 >= s.s0 && s1 <= pb.n_tokens && s.len >= 0 &&
       (long long)s.len <= ((long long)pb.table_width << p_shift);
  s.n = ok ? s1 - s.s0 : 0;
  if (!ok) s.s0 = s.len = 0;
  return s;
}

// e4m3 block scale: the smallest power of two s with amax <= 448 s, and 1 / s
// (both exact); 0 and 0 for a block below 2^-100.
__device__ __forceinline__ void pow2_scale(float amax, float& scale, float& inv) {
  if (amax < 0x1p-100f) {
    scale = inv = 0.0f;
    return;
  }
  const uint32_t u = __float_as_uint(amax);
  // amax = 1.f * 2^e and 448 = 1.75 * 2^8: s = 2^(e - 8), or 2^(e - 7) when 1.f > 1.75
  const int k = (int)(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
  scale = __uint_as_float((uint32_t)(k + 127) << 23);
  inv = __uint_as_float((uint32_t)(127 - k) << 23);
}

// A position's table row before its bounds are applied; saturating, as positions
// are any 32-bit numbers.
__device__ __forceinline__ int table_row(int pos, int pos_min) {
  int r;
  asm("sub.sat.s32 %0, %1, %2;" : "=r"(r) : "r"(pos), "r"(pos_min));
  return r;
}

// (cos, sin) of RoPE pair p at the positions pos_row[0 .. n_axes - 1]; out-of-range
// positions are clamped and flagged.
__device__ __forceinline__ float2 rope_cs(const PagedView& pv, const int32_t* pos_row, int p, bool& bad) {
  int a = 0;
  if (pv.n_axes > 1 && p >= pv.pair_off[1]) a = 1;
  if (pv.n_axes > 2 && p >= pv.pair_off[2]) a = 2;
  const int idx = table_row(pos_row[a], pv.pos_min[a]), at = max(0, min(idx, pv.pos_count[a] - 1));
  bad = bad || at != idx;
  return __ldg(pv.rope[a] + (size_t)at * pv.axis_pairs[a] + p - pv.pair_off[a]);
}

// The eight RoPE pairs p0 .. p0 + 7 that one thread rotates for many tokens.
// Where they lie in one axis at an even place (axes of a multiple of 16
// channels), a token's (cos, sin) are four 16-byte loads at one table row;
// else eight single ones.
struct RopeLane {
  const float2* row0;   // null: the pairs span axes, or start at an odd place
  int axis, stride, pos_min, last, p0;
};

__device__ __forceinline__ RopeLane rope_lane(const PagedView& pv, int p0) {
  RopeLane r;
  r.p0 = p0;
  r.axis = 0;
  if (pv.n_axes > 1 && p0 >= pv.pair_off[1]) r.axis = 1;
  if (pv.n_axes > 2 && p0 >= pv.pair_off[2]) r.axis = 2;
  const int j0 = p0 - pv.pair_off[r.axis];
  r.stride = pv.axis_pairs[r.axis];
  r.pos_min = pv.pos_min[r.axis];
  r.last = pv.pos_count[r.axis] - 1;
  r.row0 = j0 + 8 <= r.stride && ((j0 | r.stride) & 1) == 0 ? pv.rope[r.axis] + j0 : nullptr;
  return r;
}

// The lane's table row (before its bounds are applied) at the positions
// pr[0 .. n_axes - 1]
__device__ __forceinline__ int rope_index(const RopeLane& r, const int32_t* pr) { return table_row(pr[r.axis], r.pos_min); }

// (cos, sin) of the lane's pairs at the positions pr[0 .. n_axes - 1], idx = rope_index
__device__ __forceinline__ void rope_load(const PagedView& pv, const RopeLane& r, const int32_t* pr, int idx,
                                          float2 (&cs)[8], bool& bad) {
  if (r.row0) {
    const int at = max(0, min(idx, r.last));
    bad = bad || at != idx;
    const float4* t = reinterpret_cast<const float4*>(r.row0 + (size_t)at * r.stride);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 v = __ldg(t + k);
      cs[2 * k] = make_float2(v.x, v.y);
      cs[2 * k + 1] = make_float2(v.z, v.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) cs[k] = rope_cs(pv, pr, r.p0 + k, bad);
  }
}

__device__ __forceinline__ void rope_load(const PagedView& pv, const RopeLane& r, const int32_t* pr, float2 (&cs)[8],
                                          bool& bad) {
  rope_load(pv, r, pr, rope_index(r, pr), cs, bad);
}

// NaN codes (e4m3 S.1111.111) of four become zeros; true where there was one.
__device__ __forceinline__ bool drop_nan_codes(uint32_t& w) {
  const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // the top bit of each NaN byte
  w &= ~((n >> 7) * 0xFFu);
  return n != 0;
}

// 8 halfs (one uint4) -> 8 fp32 (exact); T picks the 16-bit type.
template <typename T>
__device__ __forceinline__ void load8_f32(uint4 u, float* x) {
  if constexpr (std::is_same_v<T, __half>) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
    bf16x8_to_f32(u, x);
  }
}

// Largest magnitude of 8 values in 16 bits, as a pair of 16-bit patterns (the
// order of non-negative bf16 or fp16 numbers is that of their bits).
__device__ __forceinline__ uint32_t max8_bits(uint4 u) {
  constexpr uint32_t A = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(u.x & A, u.y & A), __vmaxu2(u.z & A, u.w & A));
}

// The power of two that queries of a row are divided by on their way to fp16:
// 2^ex <= amax < 2^(ex + 1) for the row's largest magnitude (m: max8_bits of all
// of it), so that what a rotation leaves is below 2 sqrt(2).
template <typename T>
__device__ __forceinline__ int query_exponent(uint32_t m) {
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  float amax;
  if constexpr (std::is_same_v<T, __half>) amax = __half2float(__ushort_as_half((unsigned short)top));
  else amax = __uint_as_float(top << 16);
  return max(-120, min(120, (int)(__float_as_uint(amax) >> 23) - 127));
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// One RoPE pair of a query: fp32, fused.
__device__ __forceinline__ float2 rope_query(float x0, float x1, float2 cs) {
  return make_float2(fmaf(x0, cs.x, -x1 * cs.y), fmaf(x0, cs.y, x1 * cs.x));
}

// Two fp32 -> packed 16-bit pair of type T, round to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    return cvt_f16x2(lo, hi);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace kvring_dev
