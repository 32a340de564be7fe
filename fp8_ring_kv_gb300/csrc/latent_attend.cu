// latent_attend: attention over the latent cache in the absorbed form, on the
// tcgen05 tensor cores, straight from the e4m3 codes.
//
//   S^T = [C; R] Q^T      keys are the MMA's rows, query rows its columns
//   P   = 2^(y - m) w     y = scale log2(e) s_t S + log2 s_t
//   O^T += C^T P          the latent's channels are the rows
// y carries the token's scale s_t as a weight on the codes that PV sums, so a
// column's maximum m is that of what it adds, and l = sum P / s_t.
//
// A cached row is key and value: its codes lie in shared memory once, as TMA
// left them (128 keys x 128 channels, 128-byte swizzle), and are read K-major by
// QK and MN-major by PV.  The products are of 8-bit numbers, exact in fp32, and
// nothing is widened: a 16-bit copy of a 128 x 576 tile would be 147 KB of shared
// memory and its conversion half of the tensor cores' time.
//
// A bf16 query has 8 bits and is the sum of two e4m3 numbers of 4, hi = e4m3(q) and
// lo = e4m3(q - hi) (fp16: three), at a power-of-two scale of its row.  e4m3's
// smallest step is 2^-9, so what is lost is below 2^-10 / 224 of the row's largest
// number.
//
// A weight has no such neighbours: beside one key with most of a row's weight
// thousands of others share the rest, each a millionth, and they are not to be lost
// together (sums of e4m3 numbers at one scale lose what is below 2^-14.8 of the
// largest: of 8,000 keys beside one of 0.9 most of the other 0.1).
//   bf16: three e5m2 numbers of 3 bits, each of what the ones before leave.  From a
//   column's largest weight, 3584 to 57344, down to 2^-16, e5m2's smallest step: off by
//   2^-9 of a weight, or 2^-17, 2^-28.8 of the largest.
//   fp16: e4m3 and e5m2 of what is left, and the same again of 256 times the rest, in
//   an accumulator of its own: 4 + 3 + 4 + 3 bits; down to 2^-21 beside a largest weight of
//   112 to 448, 2^-27.8 of it.
//
// 64 query rows of an item, or 32 (fp16's three parts; and calls of at most 32 rows a
// sequence, where half of 64 would be empty: single tokens of 20 to 32 heads).  More
// would take the tensor memory that S needs, O of 512 channels being 64 columns a
// chunk of 128 channels.
//
// What bounds it: an instruction of 128 rows takes some 60 cycles whatever its
// columns up to 128, 66 of them a tile of 64 query rows (18 QK, 48 PV): 4,000 cycles.
// The tile takes 5,600: the next but one is loaded (2,900 cycles) only once PV has left
// its stage, the softmax (2,200) overlaps one tile's products, and its warps wait for the
// first part's (1,300) to put the third in its room: shared memory has no other.  64
// contexts of 200 to 8,000, 64 heads: 84 us; 2 of 100,000 to 131,000, 128 heads: 105 us
// (0.60 PFLOP/s of attention, 1.5 in products of codes); 9 chunks of 2 to 131 tokens, 32
// heads, window 1,024: 119 us.  (With two e4m3 parts a weight, which lost small ones: 72,
// 88 and 103.)
//
// Warp roles (640 threads, registers moved from the last group to the softmax):
//   warps 0-15  softmax: a key per thread, of a quarter of the columns (warp / 4);
//               they also rotate and split the queries and write the output
//   warp 16     MMA issue; rows of a tile that no query sees become zeros here
//   warp 17     the line of work, and TMA of the codes
#include "latent_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int LKT = 128;                     // keys of a tile
constexpr int LSOFT = 16;                    // softmax warps
constexpr int LTHREADS = 32 * (LSOFT + 4);  // (whole groups of four warps)
constexpr int kLatSoftRegs = 104, kLatOtherRegs = 64;   // per thread
// Of the sharing of work (Share): what an item costs beside its tiles (queries and
// results, 16,000 cycles), in tiles (with 3: even); units of a stretch at least; from what
// a cut is worth it (chunks over windows 120 us; with 8: 120 to 122).
constexpr int LFIX = 4, LLEAST = 6, LCUT = 4;
// A column's largest weight starts at 1/16 of its first part's largest number, 57344 of
// e5m2 (fp16: 1/4 of 448, e4m3's), and may reach that before its maximum is raised.  A higher
// start has less below the smallest steps and is raised more often (24 contexts of 300 to
// 5,000, 20 heads, fp16: 38 us, from 1/16 36).
template <typename T> constexpr float kTop = std::is_same_v<T, __half> ? 6.807354922f : 11.807354922f;
template <typename T> constexpr float kLatMost = std::is_same_v<T, __half> ? 8.807354922f : 15.807354922f;
constexpr float kRestScale = 256.0f;         // of an fp16 column's second accumulator
constexpr float kNoMax = -3.402823466e38f;   // no key yet: below every logit

struct LatStretch {
  int b, s0, n, len, lo, hi, all_lo, all_hi, k0, k1, tile, flags;
};
enum : int { LST_SOME = 1, LST_WHOLE = 2, LST_HEAD = 4 };

template <typename T, int R>
struct LatLayout {
  static constexpr bool HALF = std::is_same_v<T, __half>;
  static constexpr int NP = HALF ? 3 : 2;                        // e4m3 parts of a query
  static constexpr int HC = R / 4;                               // columns of a softmax warp
  static constexpr int CB = LKT * 128, RB = LKT * kLatRope;      // a chunk of 128 channels, the rotated part
  static constexpr int STAGE = 4 * CB + RB;
  static constexpr int QC = NP * R * 128;                        // a chunk of the queries, all parts
  static constexpr int K = 0;                                    // [2 stages]
  static constexpr int Q = K + 2 * STAGE;                        // (then the outputs on their way)
  // Weights: 64 bytes a key where the rotated part was (QK is done with it): 64
  // columns' first part, and their third once that is used; or 32 columns' two first
  // parts (fp16: of either accumulator).  The others':
  static constexpr int P = Q + 4 * QC + NP * R * kLatRope;
  static constexpr int PB = R == 64 || HALF ? LKT * 64 : LKT * 32;
  static constexpr int TOP = P + PB;                             // [4][4][HC] column maxima, sums
  static constexpr int MINE = TOP + LSOFT * HC * 4;              // [warps][HC] reference - kTop; 1 / l
  static constexpr int FAC = MINE + LSOFT * HC * 4;                  // [R] logit factors
  static constexpr int HI = FAC + R * 4;                         // [R] keys below are seen
  static constexpr int FLAG = HI + R * 4;                        // [2][16]
  static constexpr int SEG = FLAG + 128;                         // [2]
  static constexpr int BAR = SEG + 2 * (int)sizeof(LatStretch);
  static constexpr int NBAR = 2 + 4 + 2 + 2 + 1 + 1 + 2 + 2 + 4 + 4 + 1 + 2;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int ALLOC = MISC + 16;
  static_assert(ALLOC <= 232448, "shared memory of a block");
  static_assert(2 * STAGE >= (kPagedMaxSeqs + 1) * 8, "the prefix sums lie in the stages at first");
  static_assert(4 * NP * R <= 512, "tensor memory: two buffers of S below column 256, four accumulators of 64 columns");
  static_assert(LSOFT * HC * 4 >= 8 * (LTHREADS / 32), "the prefix sums' warps lie in TOP and MINE at first");
  static_assert(R == 64 ? !HALF : R == 32, "weights' room");
};

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ uint64_t sdesc_sw32(uint32_t addr, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1u << 46 |
         (uint64_t)6u << 61;
}

// Two fp16 -> packed e4m3x2, round to nearest even, saturating.
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}

// The next e4m3 part of two fp16 numbers, which keep the rest.
__device__ __forceinline__ uint32_t split2(uint32_t& v) {
  const uint32_t c = cvt_e4m3x2_f16x2(v);
  const uint32_t back = cvt_e4m3x2_to_f16x2((uint16_t)c);
  const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&back));
  v = *reinterpret_cast<const uint32_t*>(&rest);
  return c;
}

// And the next e5m2 part: an e5m2 number is the upper byte of an fp16 number.
__device__ __forceinline__ uint32_t cvt_e5m2x2_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t split2_wide(uint32_t& v) {
  const uint32_t c = cvt_e5m2x2_f16x2(v);
  const uint32_t back = __byte_perm(c, 0, 0x1404);
  const __half2 rest = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&back));
  v = *reinterpret_cast<const uint32_t*>(&rest);
  return c;
}

// What fp16 numbers v leave of x0 and x1, to be added to what the first part leaves of v:
// the parts of an fp16 query or weight have more bits than fp16 (its rounding alone was as
// much as that of an fp16 output).  Those of bf16 have fewer, and go by way of fp16 as it is.
__device__ __forceinline__ uint32_t left_of(uint32_t v, float x0, float x1) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return cvt_f16x2(x0 - f.x, x1 - f.y);
}
__device__ __forceinline__ void add_left(uint32_t& v, uint32_t left) {
  const __half2 sum = __hadd2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&left));
  v = *reinterpret_cast<const uint32_t*>(&sum);
}

// A query row's scale and 1 / scale: pow2_scale's as far down as both are normal numbers
// (smaller queries are no zeros yet: a large softmax scale may follow).
__device__ __forceinline__ void query_scale(float amax, float& scale, float& inv) {
  if (amax < 0x1p-118f) {
    scale = 0x1p-126f;
    inv = 0x1p126f;
    return;
  }
  const uint32_t u = __float_as_uint(amax);
  const uint32_t e = (u >> 23) - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7);   // 448 = 1.75 x 2^8
  scale = __uint_as_float(e << 23);
  inv = __uint_as_float((254 - e) << 23);
}

__device__ __forceinline__ float warp_maxf(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t at, uint32_t (&r)[N]) {
  if constexpr (N == 32) tmem_ld_32x32b_x32(at, r);
  else if constexpr (N == 16) tmem_ld_32x32b_x16(at, r);
  else if constexpr (N == 8) tmem_ld_32x32b_x8(at, r);
  else tmem_ld_32x32b_x4(at, r);
}

__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Ask for a line of memory to be brought to the L2.
__device__ __forceinline__ void l2_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }

// Whether one of the 128 threads at named barrier ``id`` says so.  A warp that
// gives up (the block's abort flag is set before) arrives once more: those that
// wait go on, and look at the flag.
__device__ __forceinline__ bool quarter_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void quarter_leave(int id) { asm volatile("barrier.cta.arrive %0, 128;" ::"r"(id) : "memory"); }

// a warp waits with one answer; what it has to write for the others is written
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

template <typename T, int R>
__global__ void __launch_bounds__(LTHREADS, 1)
    latent_attend_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                         const __grid_constant__ LatentAttn la) {
  using LY = LatLayout<T, R>;
  constexpr int NP = LY::NP, HC = LY::HC;
  using SH = Share<R, LKT, LFIX, 0, 0x7FFFFFFF, LLEAST, LCUT>;
  constexpr uint32_t TM_O = 256;           // four accumulators of 64 columns
  extern __shared__ __align__(1024) uint8_t sm[];
  const PagedAttn& a = la.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR);
  uint64_t* full = bars;                   // [2 stages] codes landed
  uint64_t* free_ = full + 2;              // [2][2 halves] every MMA is done with chunks 0 and 1; with all (PV is done)
  uint64_t* s_full = free_ + 4;            // [2] QK done
  uint64_t* p_full = s_full + 2;           // [2] P stored
  uint64_t* q_full = p_full + 2;           // queries written (once per stretch)
  uint64_t* q_free = q_full + 1;           // their room is free: the outputs before have left it
  uint64_t* seg_full = q_free + 1;         // [2] stretch written
  uint64_t* seg_free = seg_full + 2;       // [2]
  uint64_t* flags_in = seg_free + 2;       // [4 quarters] the warps' flags written
  uint64_t* tops_in = flags_in + 4;        // [4 quarters] their maxima, or sums, or outputs
  uint64_t* drain = tops_in + 4;
  uint64_t* first_done = drain + 1;        // (64 rows) PV is done with the weights' first part
  uint64_t* third_full = first_done + 1;   // and their third stored in its room
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC + 4);
  volatile LatStretch* segs = reinterpret_cast<volatile LatStretch*>(sm + LY::SEG);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // (the same in all lanes, for the compiler too)
  long long* warp_sums = reinterpret_cast<long long*>(sm + LY::TOP);           // at first
  unsigned long long* item_sums = reinterpret_cast<unsigned long long*>(sm + LY::MINE);
  LineOfWork* line = reinterpret_cast<LineOfWork*>(sm + LY::FAC);
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&free_[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], LSOFT);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_free[i], LSOFT + 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&flags_in[i], 4);
      mbar_init(&tops_in[i], 4);
    }
    for (int i = 0; i < 3; ++i) item_sums[i] = 0;
    mbar_init(q_full, LSOFT);
    mbar_init(q_free, LSOFT);
    mbar_init(drain, 1);
    mbar_init(first_done, 1);
    mbar_init(third_full, LSOFT);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == LSOFT) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == LSOFT + 1 && lane == 0) {
    tma_prefetch_desc(&tmC);
    tma_prefetch_desc(&tmR);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  long long* pre = reinterpret_cast<long long*>(sm + LY::K);
  const Cut cut = latent_prefix<SH, R, LKT, LTHREADS>(a, pre, warp_sums, blockIdx.x == 0, item_sums, gridDim.x, line);
  const int G = a.pv.G, C = a.pv.D, NC = C >> 7;
  const long long total = pre[a.pb.n_seqs];
  long long stretch = quotient(total + gridDim.x - 1, gridDim.x);
  if (stretch < SH::kLeast) stretch = SH::kLeast;
  if (cut.pad) stretch = cut.stretch;
  const int worker = blockIdx.x;
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  Place pl;
  if (warp == LSOFT + 1 && u < end) pl = find_place<SH, R, LKT>(a, pre, u, cut.pad);
  // the prefix sums' room is the stages' now: TMA writes there
  fence_proxy_async_smem();
  __syncthreads();

  if (warp < LSOFT) {
    // ======================================================== softmax
    reg_inc<kLatSoftRegs>();
    const int quad = warp & 3, quarter = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    float* tops = reinterpret_cast<float*>(sm + LY::TOP) + quarter * 4 * HC;   // [4][HC]
    float* mine = reinterpret_cast<float*>(sm + LY::MINE) + warp * HC;
    float* fac = reinterpret_cast<float*>(sm + LY::FAC);
    int* his = reinterpret_cast<int*>(sm + LY::HI);
    volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(sm + LY::FLAG);
    const int key_row = 32 * quad + lane;
    uint32_t n_tops = 0, n_flags = 0, n_q = 0;   // phases of their barriers so far
    int done = 0;
    bool ok = true;
    // every warp of the quarter puts HC numbers (lane c the one of column c) into tops
    auto meet = [&]() -> bool {
      warp_arrive(&tops_in[quarter]);
      return bar_warp_wait(&tops_in[quarter], n_tops++ & 1, abort_flag);
    };
    auto share = [&](float v) -> bool {
      if (lane < HC) tops[quad * HC + lane] = v;
      return meet();
    };
    auto pv_done = [&](int g) -> bool { return bar_warp_wait(&free_[(g & 1) * 2 + 1], (g >> 1) & 1, abort_flag); };
    for (int sg = 0; ok; ++sg) {
      if (!bar_warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
      const volatile LatStretch& seg = segs[sg & 1];
      const int flags = seg.flags;
      if (!(flags & LST_SOME)) break;
      const int k0 = seg.k0, n = seg.k1 - k0, s0 = seg.s0, len_n = seg.len - seg.n, seq = seg.b;
      const int lo = seg.lo, hi = seg.hi, all_lo = seg.all_lo, all_hi = seg.all_hi;
      const int r0 = seg.tile * R, rows = min(R, seg.n * G - r0);
      float l[HC];
#pragma unroll
      for (int c = 0; c < HC; ++c) l[c] = 0.0f;
      if (lane < HC) mine[lane] = kNoMax;
      if (n > 0) {
        // ------------------------------------------------------ queries
        constexpr int RW = R / LSOFT;      // rows of a warp
        const int w0 = warp * RW;
        const bool mine16 = lane * 16 < C; // lane l: latent numbers 16 l .. 16 l + 15 of every row
        uint4 w[RW][2];
        {
          int i = (r0 + w0) / G, h = r0 + w0 - i * G;
#pragma unroll
          for (int k = 0; k < RW; ++k) {
            w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
            if (w0 + k < rows && mine16) {
              const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (s0 + i) * la.q.token +
                                                                h * la.q.head) + 2 * lane;
              w[k][0] = src[0];
              w[k][1] = src[1];
            }
            if (++h >= G) {
              h = 0;
              ++i;
            }
          }
        }
        // the rotated parts of all of them: four lanes a row, 16 numbers each
        float y[16];
        uint32_t ytop = 0;
        {
          const int r = w0 + (lane >> 2), q = lane & 3;
          const bool on = (lane >> 2) < RW && r < rows;
          const int rr = r0 + (on ? r : 0), i = rr / G, h = rr - i * G;
          uint4 a0 = {}, a1 = {};
          if (on) {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(la.q_rope) + (s0 + i) * la.qr.token +
                                                              h * la.qr.head) + 2 * q;
            a0 = src[0];
            a1 = src[1];
          }
          bool bad = false;
          float2 cs[8];
          rope_load(a.pv, rope_lane(a.pv, 8 * q), a.q_pos + (size_t)(s0 + i) * a.pv.n_axes, cs, bad);
          if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
          load8_f32<T>(a0, y);
          load8_f32<T>(a1, y + 8);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float2 t = rope_query(y[2 * m], y[2 * m + 1], cs[m]);
            y[2 * m] = t.x;
            y[2 * m + 1] = t.y;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) ytop = max(ytop, __float_as_uint(y[e]) & 0x7FFFFFFFu);
          ytop = max(ytop, __shfl_xor_sync(0xFFFFFFFFu, ytop, 1));
          ytop = max(ytop, __shfl_xor_sync(0xFFFFFFFFu, ytop, 2));
        }
        // the outputs before have left the room
        bulk_wait_read();
        warp_arrive(q_free);
        if (!bar_warp_wait(q_free, n_q & 1, abort_flag)) break;
        if (tid < R) {
          // rows past the last: as the last one, with a factor of 0
          const int i = (r0 + min(tid, rows - 1)) / G;
          his[tid] = a.causal ? len_n + i + 1 : seg.len;
        }
        // x * inv in parts: 16 codes of each to ``at`` + part * ``step``
        auto put = [&](const float* x, float inv, uint8_t* at, int step) {
          uint32_t v[8], left[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = cvt_f16x2(x[2 * e] * inv, x[2 * e + 1] * inv);
            if (NP == 3) left[e] = left_of(v[e], x[2 * e] * inv, x[2 * e + 1] * inv);
          }
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            uint32_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t c0 = split2(v[2 * e]), c1 = split2(v[2 * e + 1]);
              c[e] = c0 | c1 << 16;
              if (NP == 3 && p == 0) {
                add_left(v[2 * e], left[2 * e]);
                add_left(v[2 * e + 1], left[2 * e + 1]);
              }
            }
            *reinterpret_cast<uint4*>(at + p * step) = make_uint4(c[0], c[1], c[2], c[3]);
          }
        };
        float yinv = 0.0f;
        uint8_t* qat = sm + LY::Q + (lane >> 3) * LY::QC + w0 * 128;
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const int r = w0 + k;
          const uint32_t mb = __vmaxu2(max8_bits(w[k][0]), max8_bits(w[k][1]));
          uint32_t top = max(mb & 0xFFFFu, mb >> 16);
          if constexpr (std::is_same_v<T, __half>) top = __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
          else top <<= 16;
          top = max(__reduce_max_sync(0xFFFFFFFFu, top), __shfl_sync(0xFFFFFFFFu, ytop, 4 * k));
          float scale, inv;
          query_scale(__uint_as_float(top), scale, inv);
          if (top >= 0x7F800000u) {        // no numbers: the row's scores are NaN by its factor
            scale = __int_as_float(0x7FC00000);
            inv = 0.0f;
            w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
            if ((lane >> 2) == k) {
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = 0.0f;
            }
          }
          if ((lane >> 2) == k) yinv = inv;
          // (a factor beyond fp32 would make NaN of products that are 0; at 2^87 a product that
          // is not leaves the others no weight either.  A NaN stays.)
          const float f = a.scale_log2 * scale;
          if (lane == k) fac[r] = r < rows ? (f > 0x1p87f ? 0x1p87f : f) : 0.0f;
          if (mine16) {
            float x[16];
            load8_f32<T>(w[k][0], x);
            load8_f32<T>(w[k][1], x + 8);
            put(x, inv, qat + k * 128 + (((lane & 7) ^ ((w0 + k) & 7)) << 4), R * 128);
          }
        }
        if ((lane >> 2) < RW) {
          const int r = w0 + (lane >> 2), q = lane & 3;
          put(y, yinv, sm + LY::Q + 4 * LY::QC + r * 64 + ((q ^ ((r >> 1) & 3)) << 4), R * 64);
        }
        fence_proxy_async_smem();
        warp_arrive(q_full);
        if (!bar_warp_wait(q_full, n_q++ & 1, abort_flag)) break;
        // ------------------------------------------------------ key tiles
        const int32_t* tab = a.pb.table + seq * a.pb.table_stride;
        auto page = [&](int j) -> int {    // of this thread's key of tile j; -1: not seen
          const int t = (k0 + j) * LKT + key_row;
          if (j >= n || t < lo || t >= hi) return -1;
          const int pg = tab[t >> a.pv.p_shift];
          return pg < 0 || pg >= a.pv.n_pages ? 0 : pg;
        };
        auto scale_of = [&](int j, int pg) -> float {
          return pg < 0 ? 1.0f : a.pv.k_scale[((size_t)pg << a.pv.p_shift) + (((k0 + j) * LKT + key_row) & (a.pv.P - 1))];
        };
        int pg1 = page(1);
        float s_next = scale_of(0, page(0));
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int g = done + j;
          float st = s_next;
          s_next = scale_of(j + 1, pg1);
          pg1 = page(j + 2);
          if (st == 0.0f) st = kLatMinScale;             // a row that was never written: zeros
          // a marked token has the scale NaN, and so y and weight, where it is seen
          const float est = __log2f(st), ist = st == st ? 1.0f / st : 0.0f;
          const int key = (k0 + j) * LKT + key_row;
          const bool edge = (k0 + j) * LKT < all_lo || (k0 + j + 1) * LKT > all_hi;
          if (!bar_warp_wait(&s_full[g & 1], (g >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          float x[HC];
          auto scores = [&]() {            // S of the codes
            uint32_t part[HC], part1[HC];
            const uint32_t at = tmem + lanes + (g & 1) * NP * R + quarter * HC;
            if constexpr (HC == 16) tmem_ld2_32x32b_x16(at, at + R, part, part1);
            else tmem_ld2_32x32b_x8(at, at + R, part, part1);
#pragma unroll
            for (int c = 0; c < HC; ++c) x[c] = __uint_as_float(part[c]) + __uint_as_float(part1[c]);
#pragma unroll
            for (int p = 2; p < NP; ++p) {
              tmem_ld_cols<HC>(tmem + lanes + (g & 1) * NP * R + p * R + quarter * HC, part);
#pragma unroll
              for (int c = 0; c < HC; ++c) x[c] += __uint_as_float(part[c]);
            }
          };
          // x becomes y minus what is in ``mine`` (raw: y itself).  y is rounded before the
          // difference, as where the maximum was taken: of large logits a fused one would
          // leave that rounding.
          auto logits = [&](bool raw) {
            const float4* f4 = reinterpret_cast<const float4*>(fac + quarter * HC);
            const float4* m4 = reinterpret_cast<const float4*>(mine);
            const float2 s2 = make_float2(st, st), e2 = make_float2(est, est);
#pragma unroll
            for (int c = 0; c < HC; c += 4) {
              const float4 f = f4[c / 4];
              float2 d0 = fma2(make_float2(x[c], x[c + 1]), mul2(make_float2(f.x, f.y), s2), e2);
              float2 d1 = fma2(make_float2(x[c + 2], x[c + 3]), mul2(make_float2(f.z, f.w), s2), e2);
              if (!raw) {
                const float4 m = m4[c / 4];
                d0 = add2(d0, make_float2(-m.x, -m.y));
                d1 = add2(d1, make_float2(-m.z, -m.w));
              }
              x[c] = d0.x;
              x[c + 1] = d0.y;
              x[c + 2] = d1.x;
              x[c + 3] = d1.y;
            }
            if (edge) {
#pragma unroll
              for (int c = 0; c < HC; ++c) {
                const int h = his[quarter * HC + c];
                if (key >= h || (a.window > 0 && key < h - a.window)) x[c] = -INFINITY;
              }
            }
          };
          scores();
          logits(false);
          float most = fmaxf(x[0], x[1]), most1 = fmaxf(x[2], x[3]);
#pragma unroll
          for (int c = 4; c < HC; c += 4) {
            most = max3f(most, x[c], x[c + 1]);
            most1 = max3f(most1, x[c + 2], x[c + 3]);
          }
          most = fmaxf(most, most1);
          const bool raise = quarter_any(1 + quarter, most > kLatMost<T>);
          if (*abort_flag) {
            ok = false;
            break;
          }
          if (raise) {
            uint32_t ups = 0;              // columns whose maximum is raised
#pragma unroll
            for (int c = 0; c < HC; ++c) ups |= x[c] > kLatMost<T> ? 1u << c : 0u;
            ups = __reduce_or_sync(0xFFFFFFFFu, ups);
            volatile uint32_t* fl = flag + (g & 1) * 16 + quarter * 4;
            if (lane == 0) fl[quad] = ups;
            warp_arrive(&flags_in[quarter]);
            if (!bar_warp_wait(&flags_in[quarter], n_flags++ & 1, abort_flag)) {
              ok = false;
              break;
            }
            ups = fl[0] | fl[1] | fl[2] | fl[3];
            // What was summed is brought to the new maximum.  Columns without a key
            // so far (all of them in a stretch's first tile) take it as it is.
            const bool fresh = __any_sync(0xFFFFFFFFu, lane < HC && (ups >> lane & 1) && mine[lane] == kNoMax);
            float top = -INFINITY;
            if (fresh) {
              scores();
              logits(true);
            }
#pragma unroll
            for (int c = 0; c < HC; ++c) {
              const float v = warp_maxf(x[c]);
              if (lane == c) top = v;
            }
            if (!share(top)) {
              ok = false;
              break;
            }
            float al = 1.0f, shift = 0.0f;
            if (lane < HC && (ups >> lane & 1)) {
              top = fmaxf(fmaxf(tops[lane], tops[HC + lane]), fmaxf(tops[2 * HC + lane], tops[3 * HC + lane])) - kTop<T>;
              const float was = mine[lane];
              shift = fresh ? top - was : top;
              mine[lane] = fresh ? top : was + top;
              al = ex2f(-shift);           // 0 for the column's first keys
            }
            __syncwarp();
            if (fresh) {
              scores();
              logits(false);
            } else {
#pragma unroll
              for (int c = 0; c < HC; ++c) x[c] -= __shfl_sync(0xFFFFFFFFu, shift, c);
            }
            if (j > 0) {
#pragma unroll
              for (int c = 0; c < HC; ++c) l[c] *= __shfl_sync(0xFFFFFFFFu, al, c);
              if (!pv_done(g - 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (uint32_t left = ups; left; left &= left - 1) {
                const int c = __ffs(left) - 1;
                const float f = __shfl_sync(0xFFFFFFFFu, al, c);
#pragma unroll
                for (int part = 0; part < 64 / R; ++part) {
                  const uint32_t at = tmem + lanes + TM_O + part * R + quarter * HC + c;
                  uint32_t o[4];
                  tmem_ld4_32x32b_x1(at, at + (NC > 1 ? 64 : 0), at + (NC > 2 ? 128 : 0), at + (NC > 3 ? 192 : 0), o);
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    if (q < NC) tmem_st_32x32b_x1(at + q * 64, __float_as_uint(__uint_as_float(o[q]) * f));
                }
              }
              tmem_st_wait();
            }
          }
          // weights, their sums, and their parts
#pragma unroll
          for (int c = 0; c < HC; c += 2) {
            x[c] = ex2f(x[c]);
            x[c + 1] = ex2f(x[c + 1]);
            const float2 t = fma2(make_float2(x[c], x[c + 1]), make_float2(ist, ist), make_float2(l[c], l[c + 1]));
            l[c] = t.x;
            l[c + 1] = t.y;
          }
          uint32_t v[HC / 2];
#pragma unroll
          for (int c = 0; c < HC / 2; ++c) v[c] = cvt_f16x2(x[2 * c], x[2 * c + 1]);
          const int swz = key_row >> 1 & 3;              // of the 16-byte units of 64
          uint8_t* in_stage = sm + LY::K + (g & 1) * LY::STAGE + 4 * LY::CB + key_row * 64;
          uint8_t* extra = sm + LY::P + key_row * (LY::PB / LKT);
          uint32_t w[4][HC / 4];                         // the parts
          if constexpr (LY::HALF) {
#pragma unroll
            for (int c = 0; c < HC / 2; ++c) {
              const uint32_t left = left_of(v[c], x[2 * c], x[2 * c + 1]);
              uint32_t part[4];
              part[0] = split2(v[c]);
              add_left(v[c], left);
              part[2] = split2_wide(v[c]);
              const __half2 up = __hmul2(*reinterpret_cast<const __half2*>(&v[c]), __float2half2_rn(kRestScale));
              v[c] = *reinterpret_cast<const uint32_t*>(&up);
              part[1] = split2(v[c]);
              part[3] = cvt_e5m2x2_f16x2(v[c]);
#pragma unroll
              for (int p = 0; p < 4; ++p) w[p][c / 2] = c & 1 ? w[p][c / 2] | part[p] << 16 : part[p];
            }
          } else {
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int c = 0; c < HC / 4; ++c) {
                const uint32_t c0 = split2_wide(v[2 * c]), c1 = split2_wide(v[2 * c + 1]);
                w[p][c] = c0 | c1 << 16;
              }
          }
          if constexpr (R == 64) {
            *reinterpret_cast<uint4*>(in_stage + ((quarter ^ swz) << 4)) = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
          } else {
            const int unit = quarter >> 1, half = 8 * (quarter & 1);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              *reinterpret_cast<uint2*>(in_stage + (((2 * p + unit) ^ swz) << 4) + half) = make_uint2(w[p][0], w[p][1]);
          }
          // PV of the tile before is done with the room that is there once
          if (g > 0 && !pv_done(g - 1)) {
            ok = false;
            break;
          }
          if constexpr (R == 64) {
            *reinterpret_cast<uint4*>(extra + ((quarter ^ swz) << 4)) = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
          } else {
            const int unit = quarter >> 1, half = 8 * (quarter & 1);
            if constexpr (LY::HALF) {
#pragma unroll
              for (int p = 0; p < 2; ++p)
                *reinterpret_cast<uint2*>(extra + (((2 * p + unit) ^ swz) << 4) + half) = make_uint2(w[2 + p][0], w[2 + p][1]);
            } else {
              *reinterpret_cast<uint2*>(extra + ((unit ^ (key_row >> 2 & 1)) << 4) + half) = make_uint2(w[2][0], w[2][1]);
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          warp_arrive(&p_full[g & 1]);
          if constexpr (R == 64) {                       // the third part where the first was
            if (!bar_warp_wait(first_done, g & 1, abort_flag)) {
              ok = false;
              break;
            }
            *reinterpret_cast<uint4*>(in_stage + ((quarter ^ swz) << 4)) = make_uint4(w[2][0], w[2][1], w[2][2], w[2][3]);
            fence_proxy_async_smem();
            warp_arrive(third_full);
          }
        }
        if (!ok) break;
      }
      done += n;
      // -------------------------------------------------------- results
      if (n > 0) {
        if (!pv_done(done - 1)) break;
        tc_fence_after();
      }
      // the columns' sums: lane c that of column c
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) {
        if (w >= HC) {
#pragma unroll
          for (int c = 0; c < HC; ++c) l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], w);
        } else {
#pragma unroll
          for (int c = 0; c < w; ++c) {
            const bool up = lane & w;
            const float give = up ? l[c] : l[c + w], keep = up ? l[c + w] : l[c];
            l[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, w);
          }
        }
      }
      if (!share(l[0])) break;
      const bool whole = flags & LST_WHOLE;
      const size_t at_row = (size_t)(2 * worker + (flags & LST_HEAD ? 1 : 0)) * kLatRows + quarter * HC;
      if (lane < HC) {
        const float sum = (tops[lane] + tops[HC + lane]) + (tops[2 * HC + lane] + tops[3 * HC + lane]);
        const float ref = mine[lane];
        if (!whole && quad == 0) a.tiles.ml[at_row + lane] = make_float2(ref == kNoMax ? -INFINITY : ref, sum);
        mine[lane] = sum != 0.0f ? 1.0f / sum : 0.0f;
      }
      __syncwarp();
      const int live = max(0, min(HC, rows - quarter * HC));   // columns of this warp
      auto out_row = [&](int c) -> T* {
        const int r = r0 + quarter * HC + c, i = r / G;
        return static_cast<T*>(a.out) + (s0 + i) * la.o.token + (r - i * G) * la.o.head;
      };
      if (n > 0) {
        // A thread has a channel of every row: whole rows by way of the queries'
        // room, 16-bit ones at once, fp32 pieces in two turns.
        uint8_t* stage = sm + LY::Q + quarter * HC * C * 2;
        constexpr int TC = HC / 2;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
          if (turn > 0 && !whole) {
            bulk_wait_read();
            if (!(ok = meet())) break;
          }
#pragma unroll 1
          for (int q = 0; q < NC; ++q) {
            const int ch = q * 128 + 32 * quad + lane;
            const uint32_t at_o = tmem + lanes + TM_O + q * 64 + quarter * HC + turn * TC;
            uint32_t o[TC];
            tmem_ld_cols<TC>(at_o, o);
            if constexpr (R == 32) {
              uint32_t o1[TC];
              tmem_ld_cols<TC>(at_o + R, o1);
#pragma unroll
              for (int c = 0; c < TC; ++c)
                o[c] = __float_as_uint(fmaf(__uint_as_float(o1[c]), LY::HALF ? 1.0f / kRestScale : 1.0f, __uint_as_float(o[c])));
            }
            if (whole) {
              T* at = reinterpret_cast<T*>(stage) + turn * TC * C + ch;
              const float* f = mine + turn * TC;
#pragma unroll
              for (int c = 0; c < TC; c += 2) {
                const uint32_t two = pack2<T>(__uint_as_float(o[c]) * f[c], __uint_as_float(o[c + 1]) * f[c + 1]);
                *reinterpret_cast<uint16_t*>(at + c * C) = (uint16_t)two;
                *reinterpret_cast<uint16_t*>(at + (c + 1) * C) = (uint16_t)(two >> 16);
              }
            } else {
              uint32_t* at = reinterpret_cast<uint32_t*>(stage) + ch;
#pragma unroll
              for (int c = 0; c < TC; ++c) at[c * C] = o[c];
            }
          }
          if (whole && turn == 0) continue;
          fence_proxy_async_smem();
          if (!(ok = meet())) break;       // the quarter's four warps have written
          if (whole) {
            const int c = quad * (HC / 4) + lane;
            if (lane < HC / 4 && c < live) bulk_store(out_row(c), stage + c * C * 2, C * 2);
          } else {
            const int c = quad * (TC / 4), m = min(TC / 4, live - turn * TC - c);   // the warp's rows, side by side
            if (lane == 0 && m > 0)
              bulk_store(a.tiles.o + (at_row + turn * TC + c) * C, stage + c * C * 4, m * C * 4);
          }
          bulk_commit();
        }
        if (!ok) break;
      } else if (whole) {
        for (int c = quad; c < live; c += 4)
          if (lane * 16 < C) {
            uint4* at = reinterpret_cast<uint4*>(out_row(c)) + 2 * lane;
            at[0] = at[1] = make_uint4(0, 0, 0, 0);
          }
      }
      tc_fence_before();
      warp_arrive(&seg_free[sg & 1]);
    }
    bulk_wait();
    if (*abort_flag) quarter_leave(1 + quarter);
  } else {
    reg_dec<kLatOtherRegs>();
    if (warp == LSOFT) {
      // ======================================================== MMA issue
      constexpr uint32_t idesc_qk = make_idesc(0, 0, 0, 0, LKT, NP * R);
      // (B e4m3, or e5m2 of 64 and of 32 columns)
      constexpr uint32_t idesc_pv4 = make_idesc(0, 0, 1, 1, 128, 64), idesc_pv5 = make_idesc(0, 1, 1, 1, 128, 64),
                         idesc_pv5_32 = make_idesc(0, 1, 1, 1, 128, 32);
      // The warp goes together: what it counts by is the same in all lanes.
      const uint32_t k_at = smem_u32(sm + LY::K), q_at = smem_u32(sm + LY::Q), p_at = smem_u32(sm + LY::P);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
      auto there = [&](uint64_t* bar, int phase) -> bool { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, phase & 1)); };
      int done = 0;
      uint32_t n_q = 0;
      bool ok = true;
      for (int sg = 0; ok; ++sg) {
        if (!bar_warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
        const volatile LatStretch& seg = segs[sg & 1];
        if (!(same(seg.flags) & LST_SOME)) break;
        const int k0 = same(seg.k0), n = same(seg.k1) - k0, lo = same(seg.lo), hi = same(seg.hi);
        if (n > 0 && !bar_warp_wait(q_full, n_q++ & 1, abort_flag)) break;
        // QK runs up to a tile ahead of PV where its codes are there in time; a PV that
        // can go goes first.
        int jq = 0, jp = 0;                  // the next of either
        bool begun = false;                  // of PV jp two parts are issued
        for (uint32_t tests = 1; jp < n; ++tests) {
          const int gp = done + jp, gq = done + jq, sp = gp & 1, stage = gq & 1;
          if (begun ? there(third_full, gp) : jp < jq && there(&p_full[sp], gp >> 1)) {
            tc_fence_after();
            const uint32_t kt = k_at + sp * LY::STAGE, o = tm + TM_O;
            const uint64_t b0 = make_sdesc_sw64(kt + 4 * LY::CB, 16, 512), b1 = make_sdesc_sw64(p_at, 16, 512);
            const uint32_t go = jp > 0;
            if (R == 64 && !begun) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < NC) warp_mma4_f8_ss<256, 128>(o + 64 * c, make_sdesc_sw128(kt + c * LY::CB, 16, 1024), b0, idesc_pv5, go);
              warp_mma_commit(first_done);
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (c < NC) warp_mma4_f8_ss<256, 128>(o + 64 * c, make_sdesc_sw128(kt + c * LY::CB, 16, 1024), b1, idesc_pv5, 1);
              begun = true;
              tests = 0;
              continue;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c >= NC) break;
              const uint64_t ad = make_sdesc_sw128(kt + c * LY::CB, 16, 1024);
              if constexpr (R == 64) {
                warp_mma4_f8_ss<256, 128>(o + 64 * c, ad, b0, idesc_pv5, 1);
              } else if constexpr (LY::HALF) {
                warp_mma4_f8_ss<256, 128>(o + 64 * c, ad, b0, idesc_pv4, go);
                warp_mma4_f8_ss<256, 128>(o + 64 * c, ad, b1, idesc_pv5, 1);
              } else {
                warp_mma4_f8_ss<256, 128>(o + 64 * c, ad, b0, idesc_pv5, go);
                warp_mma4_f8_ss<256, 64>(o + 64 * c, ad, sdesc_sw32(p_at, 256), idesc_pv5_32, 1);
              }
              if (c == 1) warp_mma_commit(&free_[sp * 2]);
            }
            if (NC == 1) warp_mma_commit(&free_[sp * 2]);
            warp_mma_commit(&free_[sp * 2 + 1]);
            begun = false;
            ++jp;
            tests = 0;
          } else if (jq < n && jq < jp + 2 && there(&full[stage], gq >> 1)) {
            const uint32_t kt = k_at + stage * LY::STAGE, d = tm + stage * NP * R;
            const int first = lo - (k0 + jq) * LKT, end = hi - (k0 + jq) * LKT;
            if (first > 0 || end < LKT) {
              // Rows that no query sees (in the first and last tile): their weights are
              // zeros, which must meet numbers.  (Pages of such rows came as zeros.)
              ok = bar_warp_wait(&full[stage], (gq >> 1) & 1, abort_flag);   // (there already: every lane has seen it)
              if (!ok) break;
              uint8_t* tile = sm + LY::K + stage * LY::STAGE;
              const int P = a.pv.P;
              auto clear = [&](int r0, int r1) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                for (int r = r0; r < r1; ++r) {
                  if (lane < 8 * NC) *reinterpret_cast<uint4*>(tile + (lane >> 3) * LY::CB + r * 128 + (lane & 7) * 16) = zero;
                  if (lane < 4) *reinterpret_cast<uint4*>(tile + 4 * LY::CB + r * 64 + lane * 16) = zero;
                }
              };
              if (first > 0) clear(first & -P, first);
              if (end < LKT) clear(end, min(LKT, (end + P - 1) & -P));
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c < NC)
                warp_mma4_f8_ss<2, 2>(d, make_sdesc_sw128(kt + c * LY::CB, 16, 1024),
                                    make_sdesc_sw128(q_at + c * LY::QC, 16, 1024), idesc_qk, c);
            warp_mma2_f8_ss<2, 2>(d, make_sdesc_sw64(kt + 4 * LY::CB, 16, 512), make_sdesc_sw64(q_at + 4 * LY::QC, 16, 512),
                                  idesc_qk, 1);
            warp_mma_commit(&s_full[stage]);
            ++jq;
            tests = 0;
          } else if ((tests & 255u) == 0) {
            if (tests >= kWaitTests) *abort_flag = 1;
            if (same(*abort_flag)) {
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        done += n;
        if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
      }
      // every MMA issued so far is done before the block releases its tensor memory
      warp_mma_commit(drain);
      mbar_wait(drain, 0, nullptr, 100000000ull);
      __syncwarp();
    } else if (warp == LSOFT + 1) {
      // ======================================================== the line of work
      PieceRec rec = {};
      const int P = a.pv.P, boxes = LKT / P;
      const bool alone = (long long)a.max_new * G <= R;    // every key is read by one item only
      const uint64_t once = l2_evict_first();
      int done = 0, sg = 0, armed = 0;                     // tiles, stretches; barriers armed
      bool ok = true;
      for (bool more = u < end; ok; ++sg) {
        if (sg >= 2 && !bar_warp_wait(&seg_free[sg & 1], ((sg - 2) >> 1) & 1, abort_flag)) break;
        int k0 = 0, k1 = 0;
        long long item_end = 0;
        if (more) {
          item_end = pl.at + pl.units;
          const int n = pl.t.t1 - pl.t.t0;
          k0 = pl.t.t0 + (int)max(0ll, min((long long)n, u - pl.at - LFIX));
          k1 = pl.t.t0 + (int)max(0ll, min((long long)n, min(end, item_end) - pl.at - LFIX));
        }
        if (lane == 0) {
          volatile LatStretch& seg = segs[sg & 1];
          if (more) {
            const bool head = u == pl.at;
            const int i0 = pl.tile * R / G, i1 = min(pl.s.n - 1, (pl.tile * R + R - 1) / G);
            seg.b = pl.b;
            seg.s0 = pl.s.s0;
            seg.n = pl.s.n;
            seg.len = pl.s.len;
            seg.lo = pl.t.lo;
            seg.hi = pl.t.hi;
            seg.all_hi = a.causal ? pl.s.len - pl.s.n + i0 + 1 : pl.s.len;
            seg.all_lo = a.window > 0 ? pl.s.len - pl.s.n + i1 - a.window + 1 : 0;
            seg.k0 = k0;
            seg.k1 = k1;
            seg.tile = pl.tile;
            seg.flags = LST_SOME | (head ? LST_HEAD : 0) | (head && end >= item_end ? LST_WHOLE : 0);
          } else {
            seg.flags = 0;
          }
          mbar_arrive(&seg_full[sg & 1]);
        }
        __syncwarp();
        if (!more) break;
        if (sg > 0 && k0 < k1)               // the queries, for when the softmax warps come to them
          for (int r = lane; r < min(R, pl.s.n * G - pl.tile * R); r += 32) {
            const int rr = pl.tile * R + r, i = rr / G, h = rr - i * G;
            const T* q = static_cast<const T*>(a.q) + (pl.s.s0 + i) * la.q.token + h * la.q.head;
            for (int c = 0; c < C; c += 64) l2_line(q + c);
            l2_line(static_cast<const T*>(la.q_rope) + (pl.s.s0 + i) * la.qr.token + h * la.qr.head);
          }
        const int32_t* tab = a.pb.table + pl.b * a.pb.table_stride;
        // lane i < boxes: the page of its keys of tile k; -1 where no query sees one
        auto page = [&](int k) -> int {
          const int key = k * LKT + lane * P;
          if (lane >= boxes || k >= k1 || key >= pl.t.hi || key + P <= pl.t.lo) return -1;
          const int pg = tab[key >> a.pv.p_shift];
          if (pg < 0 || pg >= a.pv.n_pages) {
            atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
            return 0;
          }
          return pg;
        };
        int pg = page(k0);
        for (int k = k0; k < k1; ++k) {
          const int g = done + k - k0, stage = g & 1;
          const int next = page(k + 1);
          // (a page that no query sees: past the last row, where TMA finds zeros)
          const int y = pg >= 0 ? (int)a.pv.row0 + (pg << a.pv.p_shift) : la.code_rows;
          uint8_t* tile = sm + LY::K + stage * LY::STAGE;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint64_t* f = &full[stage];
            if (g >= 2 && !bar_warp_wait(&free_[stage * 2 + h], ((g - 2) >> 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            const int c1 = min(NC, 2 * h + 2), chunks = max(0, c1 - 2 * h);
            if (lane == 0) mbar_arrive_expect_tx(f, LKT * (chunks * 128 + h * kLatRope));
            __syncwarp();
            if (lane < boxes) {
              for (int c = 2 * h; c < c1; ++c) {
                uint8_t* dst = tile + c * LY::CB + lane * P * 128;
                if (alone) tma_load_2d_hint(dst, &tmC, f, c * 128, y, once);
                else tma_load_2d(dst, &tmC, f, c * 128, y);
              }
              if (h == 1) {
                uint8_t* dst = tile + 4 * LY::CB + lane * P * kLatRope;
                if (alone) tma_load_2d_hint(dst, &tmR, f, C, y, once);
                else tma_load_2d(dst, &tmR, f, C, y);
              }
            }
            armed = g * 2 + h + 1;
          }
          if (!ok) break;
          pg = next;
        }
        done += k1 - k0;
        if (u == pl.at && end < item_end)
          rec = {min(pl.s.n * G - pl.tile * R, R), (int)quotient(item_end - 1, stretch), 0, pl.s.s0, pl.tile * R};
        u = min(end, item_end);
        more = u < end && next_place<SH, R, LKT>(a, pl, cut.pad);
      }
      if (lane == 0) a.tiles.rec[worker] = rec;
      // After an abort: copies still in flight land in this block's shared memory.  A
      // tile whose second half was not asked for is completed by an arrival.
      if (*abort_flag && armed > 0) {
        const int g = (armed - 1) >> 1;
        if (lane == 0 && (armed & 1)) mbar_arrive(&full[g & 1]);
        __syncwarp();
        for (int t = max(0, g - 1); t <= g; ++t) mbar_wait(&full[t & 1], (t >> 1) & 1, nullptr, 100000000ull);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&a.pv.state[PST_ERR], DEVERR_TIMEOUT);
  if (warp == LSOFT) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- joining
// The items that several blocks share (see paged_join), of either form: a warp
// per row and 128 channels, the pieces in the workers' order.
constexpr int kLatJoinWarps = 8, kLatJoinBlocks = 4;      // blocks of an SM
static_assert(32 * kLatJoinWarps >= kPagedMaxSms, "a thread per worker");
struct JoinSum {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float2 ml, const float4& x) {
    const bool some = ml.x != -INFINITY;                  // else x was not written
    const float mn = some ? fmaxf(m, ml.x) : m;
    const float f0 = mn > m ? ex2f(m - mn) : 1.0f, f1 = some ? ex2f(ml.x - mn) : 0.0f;
    m = mn;
    l = l * f0 + (some ? ml.y * f1 : ml.y);               // no key: 0; scores all NaN: NaN
    if (some) {
      o.x = o.x * f0 + x.x * f1;
      o.y = o.y * f0 + x.y * f1;
      o.z = o.z * f0 + x.z * f1;
      o.w = o.w * f0 + x.w * f1;
    }
  }
};

// What a row's sum holds -> out
template <typename T>
__device__ __forceinline__ void join_store(const PagedAttn& a, const Strides& out, const PieceRec& it, int r, int c,
                                           const JoinSum& s) {
  const float inv = s.l != 0.0f ? 1.0f / s.l : 0.0f;
  const int rr = it.row0 + r, i = rr / a.pv.G, h = it.h * a.pv.G + rr - i * a.pv.G;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (it.s0 + i) * out.token + h * out.head + c) =
      make_uint2(pack2<T>(s.o.x * inv, s.o.y * inv), pack2<T>(s.o.z * inv, s.o.w * inv));
}

// Many items, of two or three pieces: blocks (worker, share of its item's rows).
template <typename T>
__global__ void __launch_bounds__(32 * kLatJoinWarps)
    latent_join_kernel(const __grid_constant__ PagedAttn a, Strides out, int slot_rows) {
  pdl_wait();
  pdl_trigger();
  const int w = blockIdx.x, lane = threadIdx.x & 31, C = a.pv.D, NC = C >> 7;
  const PieceRec it = a.tiles.rec[w];
  for (int id = blockIdx.y * kLatJoinWarps + (threadIdx.x >> 5); id < it.rows * NC; id += gridDim.y * kLatJoinWarps) {
    const int r = id / NC, c = (id - r * NC) * 128 + lane * 4;
    JoinSum s = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll 8
    for (int p = w; p <= it.last; ++p) {
      const size_t row = (size_t)(2 * p + (p == w ? 1 : 0)) * slot_rows + r;
      s.add(a.tiles.ml[row], *reinterpret_cast<const float4*>(a.tiles.o + row * C + c));
    }
    join_store<T>(a, out, it, r, c, s);
  }
}

// Few items, of many pieces: their rows are dealt out over one wave of blocks, and up
// to 8 warps have a share of a row's pieces each.
template <typename T>
__global__ void __launch_bounds__(32 * kLatJoinWarps, kLatJoinBlocks)
    latent_join_few_kernel(const __grid_constant__ PagedAttn a, Strides out, int slot_rows, int workers) {
  __shared__ int upto[32 * kLatJoinWarps], sums[kLatJoinWarps];   // rows x chunks of the workers up to here
  __shared__ float4 part_o[kLatJoinWarps][32];
  __shared__ float2 part_ml[kLatJoinWarps];
  __shared__ PieceRec recs[32 * kLatJoinWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, C = a.pv.D, NC = C >> 7;
  int n = 0;
  if (tid < workers) {
    recs[tid] = a.tiles.rec[tid];
    n = recs[tid].rows * NC;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, n, d);
    if (lane >= d) n += v;
  }
  if (lane == 31) sums[warp] = n;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int i = 0; i < kLatJoinWarps; ++i) {
    if (i < warp) n += sums[i];
    total += sums[i];
  }
  upto[tid] = n;
  __syncthreads();
  int bits = 0;                            // 2^bits warps of a row
  while ((1 << bits) < kLatJoinWarps && (total << (bits + 1)) <= (int)gridDim.x * kLatJoinWarps) ++bits;
  const int split = 1 << bits, groups = kLatJoinWarps >> bits, part = warp & (split - 1);
  for (int first = blockIdx.x * groups; first < total; first += gridDim.x * groups) {
    const int id = first + (warp >> bits);
    JoinSum s = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    PieceRec it = {};
    int r = 0, c = 0;
    if (id < total) {
      int w = 0;
#pragma unroll
      for (int i = 0; i < kLatJoinWarps; ++i) w += __popc(__ballot_sync(0xFFFFFFFFu, upto[32 * i + lane] <= id));
      const int at = id - (w > 0 ? upto[w - 1] : 0);
      it = recs[w];
      r = at / NC;
      c = (at - r * NC) * 128 + lane * 4;
      const int pieces = it.last - w + 1;
      const int end = w + (pieces * (part + 1) >> bits);
#pragma unroll 1
      for (int p = w + (pieces * part >> bits); p < end; p += 4) {
        float2 ml[4];
        float4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {      // (all loads on their way at once)
          const size_t row = (size_t)(2 * (p + k) + (p + k == w ? 1 : 0)) * slot_rows + r;
          ml[k] = p + k < end ? a.tiles.ml[row] : make_float2(-INFINITY, 0.0f);
          x[k] = p + k < end ? *reinterpret_cast<const float4*>(a.tiles.o + row * C + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) s.add(ml[k], x[k]);
      }
    }
    if (split > 1) {                       // (one turn of the loop)
      part_o[warp][lane] = s.o;
      if (lane == 0) part_ml[warp] = make_float2(s.m, s.l);
      __syncthreads();
      if (part > 0 || id >= total) continue;
      for (int i = 1; i < split; ++i) s.add(part_ml[warp + i], part_o[warp + i][lane]);
    }
    if (id < total) join_store<T>(a, out, it, r, c, s);
  }
}

// ---------------------------------------------------------------- host
static size_t piece_bytes(int rows, int width) {
  const size_t slots = (size_t)2 * kPagedMaxSms * rows;
  return slots * width * 4 + slots * 8 + kPagedMaxSms * sizeof(PieceRec);
}

size_t latent_scratch_bytes(int C) {
  const size_t a = piece_bytes(kLatRows, C), b = piece_bytes(kTilesRows, kLatHead);
  return a > b ? a : b;
}

void latent_carve_scratch(uint8_t* base, int rows, int width, PagedAttn* a) {
  const size_t slots = (size_t)2 * kPagedMaxSms * rows;
  a->tiles.o = reinterpret_cast<float*>(base);
  a->tiles.ml = reinterpret_cast<float2*>(base + slots * width * 4);
  a->tiles.rec = reinterpret_cast<PieceRec*>(base + slots * width * 4 + slots * 8);
}

template <typename T>
static cudaError_t join_t(const PagedAttn& a, const Strides& o, int slot_rows, int rows, int blocks, cudaStream_t st) {
  const dim3 block(32 * kLatJoinWarps);
  // No more items than this.  With four pieces each or more the rows of the few are
  // dealt out (2 items of 128 heads: 8 us less); with fewer pieces the search for a row
  // costs more than it gives (40 items, 9 chunks in 152: 3 to 5 us more).
  const long long G = a.pv.G, by_seq = a.pb.n_seqs * ((a.max_new * G + rows - 1) / rows),
                  by_row = a.pb.n_seqs + a.pb.n_tokens * G / rows;
  if ((by_seq < by_row ? by_seq : by_row) * a.pv.H * 4 <= blocks)
    return launch_pdl(latent_join_few_kernel<T>, dim3(blocks * kLatJoinBlocks), block, 0, st, a, o, slot_rows, blocks);
  const int shares = (rows * (a.pv.D >> 7) + kLatJoinWarps - 1) / kLatJoinWarps;
  return launch_pdl(latent_join_kernel<T>, dim3(blocks, shares), block, 0, st, a, o, slot_rows);
}

cudaError_t launch_latent_join(const PagedAttn& a, const Strides& o, int slot_rows, int rows, bool f16, int blocks,
                               cudaStream_t st) {
  return f16 ? join_t<__half>(a, o, slot_rows, rows, blocks, st) : join_t<__nv_bfloat16>(a, o, slot_rows, rows, blocks, st);
}

template <typename T, int R>
static cudaError_t prepare_t() {
  // reg_inc draws on the registers that the block was launched with: fewer
  // would make it wait for ever
  cudaFuncAttributes fa;
  const cudaError_t e = cudaFuncGetAttributes(&fa, latent_attend_kernel<T, R>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * LTHREADS < 32 * (LSOFT * kLatSoftRegs + 4 * kLatOtherRegs)) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(latent_attend_kernel<T, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              LatLayout<T, R>::ALLOC);
}

cudaError_t prepare_latent_attend() {
  cudaError_t e = prepare_t<__half, 32>();
  if (e == cudaSuccess) e = prepare_t<__nv_bfloat16, 32>();
  if (e == cudaSuccess) e = prepare_t<__nv_bfloat16, 64>();
  return e;
}

template <typename T, int R>
static cudaError_t attend_t(const LatentAttn& la, const CUtensorMap& tmC, const CUtensorMap& tmR, int blocks,
                            cudaStream_t st) {
  const cudaError_t e = launch_pdl(latent_attend_kernel<T, R>, dim3(blocks), dim3(LTHREADS), LatLayout<T, R>::ALLOC, st,
                                   tmC, tmR, la);
  return e == cudaSuccess ? launch_latent_join(la.a, la.o, kLatRows, R, std::is_same_v<T, __half>, blocks, st) : e;
}

cudaError_t launch_latent_attend(const LatentAttn& la, const CUtensorMap& tmC, const CUtensorMap& tmR, bool f16, int sms,
                                 cudaStream_t st) {
  const int blocks = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  if (f16) return attend_t<__half, 32>(la, tmC, tmR, blocks, st);
  // (items of 32 rows and of 64: one token of 32 heads over 900 34 and 47 us, 32 over
  // 1,000 to 4,000 42 and 54)
  if ((long long)la.a.max_new * la.a.pv.G <= 32) return attend_t<__nv_bfloat16, 32>(la, tmC, tmR, blocks, st);
  return attend_t<__nv_bfloat16, 64>(la, tmC, tmR, blocks, st);
}

}  // namespace kvring_dev
