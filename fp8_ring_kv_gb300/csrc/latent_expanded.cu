// latent_expanded: attention with keys and values of every head, 128 numbers of
// its own and a rotated key part of 64 that the heads share, on the tcgen05
// tensor cores.
//
//   S = [Q, rope(Qr)] [K; Kr]^T    kind::f16, the inputs' own type
//   P = 2^(y - m + 6), 16 bits, in tensor memory over the S it came from
//   O += P V                       A = P from tensor memory
//
// A block works on two tiles of 128 query rows of one head over the same keys:
// while the softmax of one runs, the tensor cores work on the other.  The shared
// key part is a third block of K's tile, read where it lies, so no head's keys
// are written out 192 wide.
//
// A weight of the inputs' type would be off by as much as the output is rounded by,
// and over many keys of like weight all of that shows (1.6 times the output's own
// rounding, with the rotated queries'; 1.3 without it): weights are the sum of two such
// numbers, two products into one O (S leaves room for both).
//
// What bounds it: the tensor pipe (128 keys of 256 rows: 24 steps of 128 x 128 x
// 16 for S and 32 for PV of each tile, 64 cycles each, 3,584); the tile takes some 5,000
// cycles, the difference mostly pauses between a PV and the
// QK that overwrites its weights (below).  512 queries over 16,001 keys, 20
// heads: 126 us (0.85 PFLOP/s of attention, 44% of what cuBLAS reaches in bf16, and
// 1.6 times that in products); 3 prompts of 1,000 to 4,096, 32 heads, causal: 357.
//
// Warp roles (640 threads, registers moved from the last group to the softmax):
//   warps 0-15   softmax: of query tile t and half p of its keys, warps 8 p + 4 t
//                .. + 3, one row per thread: two warps share a row.  They also load
//                and rotate the queries and write the output
//   warp 16      MMA issue
//   warp 17      the line of work, and TMA
//   warps 18, 19 values that not every row sees: those that no row sees become
//                zeros, a NaN or infinity that some see is taken out (its weight in the
//                others is 0, which must meet a number) and remembered
// QK of the next tile overwrites the P that PV of this one reads, with another
// accumulator: products of different accumulators have no documented order, so
// it is issued once that PV has completed.
#include "latent_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int XKT = 128, XROWS = 128, XTR = kTilesRows, XTHREADS = 640;
static_assert(XTR == 2 * XROWS);
constexpr int kXSoftmaxRegs = 104, kXOtherRegs = 64;   // per thread: 16 warps and 4
// Of the sharing of work (Share): what an item costs beside its tiles (queries and
// results, 15,000 cycles), in tiles (3 prompts of 1,000 to 4,096, 32 heads: 353 us;
// with 2: 382, with 8: 368); units of a stretch at least; and from what a cut is worth
// it (2 sequences of 100 to 2,000 over 3,000: 64 us, with 8: 73).
constexpr int XFIX = 5, XLEAST = 6, XCUT = 3;
constexpr int XRING = 8, XBLK = 16384;       // blocks of K (128 keys x 64 numbers) and V (64 keys x 128)
constexpr float kXRaise = 8.0f;              // a row's maximum is raised when a tile exceeds it by 2^8 ...
constexpr float kXTop = 6.0f;                // ... and starts its weights at 2^6, so they stay below 2^14 in fp16

struct XStretch {
  int s0, n, len, lo, hi, all_lo, all_hi, k0, k1, tile, h, key0, flags;
};
enum : int { XST_SOME = 1, XST_WHOLE = 2, XST_HEAD = 4, XST_SKIP = 8 };

struct XLayout {
  static constexpr int QT = 3 * XROWS * 128;             // a query tile: three blocks of 64 numbers
  static constexpr int Q = 0;
  static constexpr int RING = Q + 2 * QT;
  static constexpr int SEG = RING + XRING * XBLK;
  static constexpr int SLOT = SEG + 2 * 64;              // [2 halves][256] a row's maxima; sums
  static constexpr int BAR = SLOT + 2 * XTR * 4;
  static constexpr int NBAR = 4 * 2 + 5 * 2 + 4 + 1 + 16 + 8;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int ALLOC = MISC + 16;
  static_assert(sizeof(XStretch) <= 64 && ALLOC <= 232448, "shared memory of a block");
  static_assert(2 * QT >= (kPagedMaxSeqs + 1) * 8, "the prefix sums lie in the query tiles at first");
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The 16-bit numbers of w that are no numbers become zeros; true where there was one.
template <typename T>
__device__ __forceinline__ bool drop_nonfinite(uint32_t& w) {
  constexpr uint32_t E = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
  const bool lo = (w & E) == E, hi = (w & (E << 16)) == (E << 16);
  if (lo) w &= 0xFFFF0000u;
  if (hi) w &= 0x0000FFFFu;
  return lo || hi;
}

// Whether one of the values of keys lo, lo + 2, .. < hi is no number, tiles that
// every row sees left out.
template <typename T>
__device__ __noinline__ bool nonfinite_among(const T* v, long long v_token, int lo, int hi, int all_lo, int all_hi) {
#pragma unroll 1
  for (int key = lo; key < hi; key += 2) {
    const int k = key / XKT;
    if (k * XKT >= all_lo && k * XKT + XKT <= all_hi) continue;
    const uint4* p = reinterpret_cast<const uint4*>(v + key * v_token);
#pragma unroll 1
    for (int c = 0; c < kLatHead / 8; ++c) {
      uint4 w = p[c];
      if (drop_nonfinite<T>(w.x) | drop_nonfinite<T>(w.y) | drop_nonfinite<T>(w.z) | drop_nonfinite<T>(w.w)) return true;
    }
  }
  return false;
}

template <typename T>
__global__ void __launch_bounds__(XTHREADS, 1)
    latent_expanded_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmR,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ExpandedAttn xa) {
  using LY = XLayout;
  using SH = Share<XTR, XKT, XFIX, 0, 0x7FFFFFFF, XLEAST, XCUT>;
  constexpr uint32_t TM_S = 0, TM_O = 256;
  constexpr uint32_t FMT = std::is_same_v<T, __half> ? 0 : 1;
  extern __shared__ __align__(1024) uint8_t sm[];
  const PagedAttn& a = xa.a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR);
  uint64_t* k_full = bars;                 // [2] (tiles in turn) K's three blocks landed
  uint64_t* v_full = k_full + 2;           // [2] V's two
  uint64_t* k_free = v_full + 2;           // [2] every MMA is done with K's blocks
  uint64_t* v_free = k_free + 2;           // [2] and with V's
  uint64_t* q_full = v_free + 2;           // [2 query tiles]
  uint64_t* s_full = q_full + 2;           // [2] QK done
  uint64_t* p_full = s_full + 2;           // [2] P stored
  uint64_t* o_done = p_full + 2;           // [2] PV done
  uint64_t* v_clean = o_done + 2;          // [2] (tiles in turn) values looked at
  uint64_t* seg_full = v_clean + 2;        // [2]
  uint64_t* seg_free = seg_full + 2;       // [2]
  uint64_t* drain = seg_free + 2;
  uint64_t* m_ready = drain + 1;           // [2][4 warps][2 halves] a half's maxima written
  uint64_t* both = m_ready + 16;           // [2][4] both warps of a row are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC + 4);
  volatile int* odd_seen = reinterpret_cast<volatile int*>(sm + LY::MISC + 8);   // a value that is no number was taken out
  auto seg_at = [&](int sg) { return reinterpret_cast<volatile XStretch*>(sm + LY::SEG + (sg & 1) * 64); };
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // (the same in all lanes, for the compiler too)
  unsigned long long* item_sums = reinterpret_cast<unsigned long long*>(sm + LY::RING);        // at first
  long long* warp_sums = reinterpret_cast<long long*>(sm + LY::RING + 64);
  LineOfWork* line = reinterpret_cast<LineOfWork*>(sm + LY::RING + 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 3);
      mbar_init(&v_full[i], 2);
      mbar_init(&k_free[i], 1);
      mbar_init(&v_free[i], 1);
      mbar_init(&q_full[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&o_done[i], 1);
      mbar_init(&v_clean[i], 2);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_free[i], 19);
    }
    for (int i = 0; i < 16; ++i) mbar_init(&m_ready[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&both[i], 2);
    mbar_init(drain, 1);
    for (int i = 0; i < 3; ++i) item_sums[i] = 0;
    *abort_flag = 0;
    *odd_seen = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 17 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmR);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  long long* pre = reinterpret_cast<long long*>(sm + LY::Q);
  const Cut cut = latent_prefix<SH, XTR, XKT, XTHREADS>(a, pre, warp_sums, blockIdx.x == 0, item_sums, gridDim.x, line);
  const long long total = pre[a.pb.n_seqs] * a.pv.H;
  long long stretch = quotient(total + gridDim.x - 1, gridDim.x);
  if (stretch < SH::kLeast) stretch = SH::kLeast;
  if (cut.pad) stretch = cut.stretch;
  const int worker = blockIdx.x;
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  Place pl;
  if (warp == 17 && u < end) pl = find_place<SH, XTR, XKT>(a, pre, u, cut.pad);
  // the prefix sums' room is the query tiles' now, the others' the ring's
  fence_proxy_async_smem();
  __syncthreads();

  if (warp < 16) {
    // ======================================================== softmax
    reg_inc<kXSoftmaxRegs>();
    const int t = (warp >> 2) & 1, par = warp >> 3, quad = warp & 3, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t s_at = tmem + lanes + TM_S + 128 * t, o_at = tmem + lanes + TM_O + 128 * t;
    float* slots = reinterpret_cast<float*>(sm + LY::SLOT) + t * XROWS + row;
    float *mine = slots + par * XTR, *other = slots + (par ^ 1) * XTR;
    const int pair = 4 * t + quad;         // the two warps of these rows
    uint32_t nb = 0, tiles = 0;            // phases of ``both``; of this query tile's barriers
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&both[pair]);
      return bar_warp_wait(&both[pair], nb++ & 1, abort_flag);
    };
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      if (!bar_warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
      const volatile XStretch& seg = *seg_at(sg);
      const int flags = seg.flags;
      if (!(flags & XST_SOME)) break;
      const int k0 = seg.k0, n = seg.k1 - k0, s0 = seg.s0, len_n = seg.len - seg.n, head = seg.h;
      const int r0 = seg.tile * XTR + t * XROWS, rows = min(XROWS, seg.n - r0);   // of this query tile
      const bool live = row < rows;
      const int i = r0 + row;
      const int hi = !live ? 0x7FFFFFFF : a.causal ? len_n + i + 1 : seg.len;
      const int lo = live && a.window > 0 ? len_n + i - a.window + 1 : 0;
      float ms = -INFINITY, m = -INFINITY, l = 0.0f;    // the reference as a score and as a logit; the sum
      if (n > 0 && rows > 0) {
        // ------------------------------------------------------ queries
        // half of the pair's 32 rows each
        uint8_t* tile = sm + LY::Q + t * LY::QT;
        const T* q = static_cast<const T*>(a.q) + (long long)(s0 + r0) * xa.q.token + (long long)head * xa.q.head;
        const int w0 = 32 * quad + 16 * par;
        const int rq = lane & 3;                         // the rotated part: 4 lanes of 16 numbers
        const RopeLane rl = rope_lane(a.pv, 8 * rq);
        bool bad = false;
#pragma unroll 1
        for (int b0 = 0; b0 < 16; b0 += 8) {
          uint4 w[4];                                    // 128 numbers of a row: 16 lanes
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = w0 + b0 + 2 * k + (lane >> 4);
            w[k] = make_uint4(0, 0, 0, 0);
            if (r < rows) w[k] = *(reinterpret_cast<const uint4*>(q + r * xa.q.token) + (lane & 15));
          }
          const int rr = w0 + b0 + (lane >> 2);
          const bool on = rr < rows;
          uint4 a0 = {}, a1 = {};
          if (on) {
            const uint4* src = reinterpret_cast<const uint4*>(q + rr * xa.q.token + kLatHead) + 2 * rq;
            a0 = src[0];
            a1 = src[1];
          }
          float2 cs[8];
          rope_load(a.pv, rl, a.q_pos + (size_t)(s0 + r0 + (on ? rr : 0)) * a.pv.n_axes, cs, bad);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = w0 + b0 + 2 * k + (lane >> 4), c = lane & 15;
            *reinterpret_cast<uint4*>(tile + (c >> 3) * (XROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[k];
          }
          float x[16];
          load8_f32<T>(a0, x);
          load8_f32<T>(a1, x + 8);
          uint32_t v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 y = rope_query(x[2 * e], x[2 * e + 1], cs[e]);
            v[e] = pack2<T>(y.x, y.y);
          }
          uint8_t* at = tile + 2 * (XROWS * 128) + rr * 128;
          *reinterpret_cast<uint4*>(at + (((2 * rq) ^ (rr & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<uint4*>(at + (((2 * rq + 1) ^ (rr & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
        }
        if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
        // ------------------------------------------------------ key tiles
        const float rf = a.scale_log2;
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++tiles) {
          if (!bar_warp_wait(&s_full[t], tiles & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t xr[64];
          tmem_ld_32x32b_x64(s_at + 64 * par, xr);
          const int key0 = (k0 + j) * XKT + 64 * par;
          if (__any_sync(0xFFFFFFFFu, key0 + 64 > hi || key0 < lo)) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (key0 + k >= hi || key0 + k < lo) xr[k] = 0xFF800000u;   // -inf
          }
          const float* s = reinterpret_cast<const float*>(xr);
          float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int k = 4; k < 60; k += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = max3f(m4[e], s[k + e], s[k + 4 + e]);
          }
          // the row's maximum: the other half's keys are the other warp's.  Both
          // see the same numbers and do the same.
          const float my = fmaxf(max3f(max3f(m4[0], s[60], s[61]), max3f(m4[1], s[62], s[63]), m4[2]), m4[3]);
          *mine = my;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_ready[2 * pair + par]);
          if (!bar_warp_wait(&m_ready[2 * pair + (par ^ 1)], tiles & 1, abort_flag)) {
            ok = false;
            break;
          }
          const float mms = fmaxf(my, *other), mm = mms * rf;
          if (__any_sync(0xFFFFFFFFu, mm > m + kXRaise)) {
            // rare after a row's first keys: what was summed is brought to the new maximum
            const float mn = mm > m + kXRaise ? mm : m;
            const float al = mn > m ? ex2f(m - mn) : 1.0f;     // 0 for the row's first keys
            if (mn > m) ms = mms;
            m = mn;
            l *= al;
            if (j > 0) {
              // QK of this tile was issued after the PV before it had completed
#pragma unroll 1
              for (int k = par * 64; k < par * 64 + 64; k += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(o_at + k, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st_32x32b_x16(o_at + k, o);
              }
            }
          }
          // (both warps hold their scores in registers: P may go over all of S)
          // Differences of scores, then their logits: of large logits the maximum's rounding
          // would show in a difference of those.
          const float from = m == -INFINITY ? 0.0f : -ms;
          float2 part[2] = {};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16], p1[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 y = fma2(add2(make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), make_float2(from, from)),
                              make_float2(rf, rf), make_float2(kXTop, kXTop));
              y.x = ex2f(y.x);
              y.y = ex2f(y.y);
              part[e & 1] = add2(part[e & 1], y);
              p[e] = pack2<T>(y.x, y.y);
              const float2 first = unpack2<T>(p[e]);
              p1[e] = pack2<T>(y.x - first.x, y.y - first.y);
            }
            tmem_st_32x32b_x16(s_at + 32 * par + 16 * c, p);
            tmem_st_32x32b_x16(s_at + 64 + 32 * par + 16 * c, p1);
          }
          l += (part[0].x + part[0].y) + (part[1].x + part[1].y);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (ok && !bar_warp_wait(&o_done[t], (tiles - 1) & 1, abort_flag)) ok = false;
        if (!ok) break;
        tc_fence_after();
        if (*odd_seen && live &&
            nonfinite_among<T>(static_cast<const T*>(xa.v) + (long long)seg.key0 * xa.v_token + (long long)head * xa.v_head,
                               xa.v_token, max(max(lo, seg.lo), k0 * XKT) + par, min(min(hi, seg.hi), (k0 + n) * XKT),
                               seg.all_lo, seg.all_hi))
          l = __int_as_float(0x7FFFFFFF);                // the row sees one of the values taken out
        // the row's sum: both halves
        *mine = l;
        if (!meet()) break;
        l = slots[0] + slots[XTR];
        if (!meet()) break;
      }
      // -------------------------------------------------------- results
      if (rows > 0 && !(flags & XST_SKIP)) {
        // half of the channels each
        const bool whole = flags & XST_WHOLE;
        const size_t at_row = (size_t)(2 * worker + (flags & XST_HEAD ? 1 : 0)) * XTR + t * XROWS + row;
        if (!whole && live && par == 0) a.tiles.ml[at_row] = make_float2(m, l);
        if (whole || n > 0) {
          const float inv = l != 0.0f ? 1.0f / l : 0.0f;
          T* dst = static_cast<T*>(a.out) + (long long)(s0 + i) * xa.o.token + (long long)head * xa.o.head;
#pragma unroll 1
          for (int c = par * 64; c < par * 64 + 64; c += 32) {
            uint32_t o[32];
            if (n > 0) {
              tmem_ld_32x32b_x32(o_at + c, o);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
            if (!live) continue;
            if (whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = pack2<T>(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                reinterpret_cast<uint4*>(dst + c)[k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                reinterpret_cast<uint4*>(a.tiles.o + at_row * kLatHead + c)[k] =
                    make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
    }
  } else {
    reg_dec<kXOtherRegs>();
    if (warp == 16) {
      // ====================================================== MMA issue
      // The warp goes together: what it counts by is the same in all lanes.
      constexpr uint32_t idesc_qk = make_idesc(FMT, FMT, 0, 0, XROWS, XKT);
      constexpr uint32_t idesc_pv = make_idesc(FMT, FMT, 0, 1, XROWS, kLatHead);
      const uint32_t q0 = smem_u32(sm + LY::Q), ring = smem_u32(sm + LY::RING);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
      uint32_t nq = 0, nq1 = 0, steps0 = 0, steps1 = 0;    // of either query tile
      int done = 0;
      bool ok = true;
      auto block = [&](int b) { return ring + (b & (XRING - 1)) * XBLK; };
      auto there = [&](uint64_t* bar, uint32_t phase) -> bool { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, phase & 1)); };
      auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {
        for (uint32_t tests = 1; !there(bar, phase); ++tests)
          if ((tests & 255u) == 0) {
            if (tests >= kWaitTests) *abort_flag = 1;
            if (same(*abort_flag)) return false;
          }
        return true;
      };
      auto qk = [&](int t, int g) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
          warp_mma4_f16_ss(tm + TM_S + 128 * t, make_sdesc_sw128(q0 + t * LY::QT + c * (XROWS * 128), 16, 1024),
                           make_sdesc_sw128(block(5 * g + c), 16, 1024), idesc_qk, c);
      };
      auto pv = [&](int t, int g, uint32_t accumulate) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          warp_mma4_f16_ts(tm + TM_O + 128 * t, tm + TM_S + 128 * t + 32 * c,
                           make_sdesc_sw128(block(5 * g + 3 + (c & 1)), XBLK / 2, 1024), idesc_pv, accumulate | c);
      };
      for (int sg = 0; ok; ++sg) {
        if (!bar_warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
        const volatile XStretch& seg = *seg_at(sg);
        if (!(same(seg.flags) & XST_SOME)) break;
        const int n = same(seg.k1) - same(seg.k0);
        const int last = same(seg.n) - same(seg.tile) * XTR > XROWS ? 1 : 0;   // the second query tile has rows
        if (n > 0) {
          ok = wait(&k_full[done & 1], done >> 1) && wait(&q_full[0], nq++);
          if (!ok) break;
          tc_fence_after();
          qk(0, done);
          warp_mma_commit(&s_full[0]);
          if (last) {
            ok = wait(&q_full[1], nq1++);
            if (!ok) break;
            tc_fence_after();
            qk(1, done);
            warp_mma_commit(&s_full[1]);
          }
          warp_mma_commit(&k_free[done & 1]);
        }
        // What a product waits for is looked at while the one before it runs: a wait
        // takes hundreds of cycles behind products even where it is over.
        bool ready = false;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int g = done + j;
#pragma unroll 1
          for (int t = 0; t <= last && ok; ++t) {
            const uint32_t step = t ? steps1 : steps0;
            if (!ready) ok = (t > 0 || wait(&v_clean[g & 1], g >> 1)) && wait(&p_full[t], step);
            if (!ok) break;
            tc_fence_after();
            pv(t, g, j > 0);
            warp_mma_commit(&o_done[t]);
            ready = false;
            if (j + 1 < n) {
              if (t == 0) ok = wait(&k_full[(g + 1) & 1], (g + 1) >> 1);
              if (t < last) ready = there(&p_full[1], steps1);
              else if (last > 0) ready = there(&v_clean[(g + 1) & 1], (g + 1) >> 1) && there(&p_full[0], steps0);
              ok = ok && wait(&o_done[t], step);
              if (!ok) break;
              if (t == last && lane == 0) mbar_arrive(&v_free[g & 1]);
              __syncwarp();
              tc_fence_after();
              qk(t, g + 1);
              warp_mma_commit(&s_full[t]);
              if (t == last) warp_mma_commit(&k_free[(g + 1) & 1]);
            }
            if (t) ++steps1;
            else ++steps0;
          }
        }
        if (ok && n > 0) ok = wait(&o_done[0], steps0 - 1);
        if (ok && n > 0 && last) ok = wait(&o_done[1], steps1 - 1);
        if (!ok) break;
        if (n > 0 && lane == 0) mbar_arrive(&v_free[(done + n - 1) & 1]);
        done += n;
        if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
      }
      // every MMA issued so far is done before the block releases its tensor memory
      warp_mma_commit(drain);
      mbar_wait(drain, 0, nullptr, 100000000ull);
      __syncwarp();
    } else if (warp == 17) {
      // ====================================================== the line of work
      PieceRec rec = {};
      int done = 0, sg = 0, armed = 0;                   // tiles, stretches; blocks armed
      bool ok = true;
      for (bool more = u < end; ok; ++sg) {
        if (sg >= 2 && !bar_warp_wait(&seg_free[sg & 1], ((sg - 2) >> 1) & 1, abort_flag)) break;
        int k0 = 0, k1 = 0, key0 = 0;
        long long item_end = 0;
        bool skip = false;
        if (more) {
          item_end = pl.at + pl.units;
          const int n = pl.t.t1 - pl.t.t0;
          k0 = pl.t.t0 + (int)max(0ll, min((long long)n, u - pl.at - XFIX));
          k1 = pl.t.t0 + (int)max(0ll, min((long long)n, min(end, item_end) - pl.at - XFIX));
          key0 = a.pb.table[pl.b];
          skip = key0 < 0 || (long long)key0 + pl.s.len > xa.n_keys;
          if (skip) {
            if (lane == 0) atomicOr(&a.pv.state[PST_ERR], DEVERR_SEQ);
            k1 = k0;
          }
        }
        if (lane == 0) {
          volatile XStretch& seg = *seg_at(sg);
          if (more) {
            const bool head = u == pl.at;
            const int i0 = pl.tile * XTR, i1 = min(pl.s.n - 1, pl.tile * XTR + XTR - 1);
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
            seg.h = pl.h;
            seg.key0 = key0;
            seg.flags = XST_SOME | (skip ? XST_SKIP : 0) | (head ? XST_HEAD : 0) | (head && end >= item_end ? XST_WHOLE : 0);
          } else {
            seg.flags = 0;
          }
          mbar_arrive(&seg_full[sg & 1]);
        }
        __syncwarp();
        if (!more) break;
        for (int k = k0; k < k1 && ok; ++k) {
          const int b0 = 5 * (done + k - k0), at = key0 + k * XKT;
          for (int c = 0; c < 5; ++c) {
            const int b = b0 + c, slot = b & (XRING - 1);
            if (b >= XRING) {              // the block that was there: K's or V's of tile o
              const int o = (b - XRING) / 5;
              if (!bar_warp_wait(((b - XRING) - 5 * o < 3 ? k_free : v_free) + (o & 1), (o >> 1) & 1, abort_flag)) {
                ok = false;
                break;
              }
            }
            if (lane == 0) {
              uint8_t* dst = sm + LY::RING + slot * XBLK;
              uint64_t* bar = (c < 3 ? k_full : v_full) + ((done + k - k0) & 1);
              mbar_arrive_expect_tx(bar, XBLK);
              if (c < 2) tma_load_3d(dst, &tmK, bar, 64 * c, at, pl.h);
              else if (c == 2) tma_load_2d(dst, &tmR, bar, 0, at);
              else
                for (int d = 0; d < 2; ++d)
                  tma_load_3d(dst + d * (XBLK / 2), &tmV, bar, 64 * d, at + 64 * (c - 3), pl.h);
            }
            __syncwarp();
            armed = b + 1;
          }
        }
        if (!ok) break;
        done += k1 - k0;
        if (u == pl.at && end < item_end && !skip)
          rec = {min(pl.s.n - pl.tile * XTR, XTR), (int)quotient(item_end - 1, stretch), pl.h, pl.s.s0, pl.tile * XTR};
        u = min(end, item_end);
        more = u < end && next_place<SH, XTR, XKT>(a, pl, cut.pad);
      }
      if (lane == 0) a.tiles.rec[worker] = rec;
      // After an abort: copies still in flight land in this block's shared memory.  A
      // tile whose blocks were not all asked for is completed by arrivals.
      if (*abort_flag && armed > 0) {
        const int g = (armed - 1) / 5, c = armed - 5 * g;     // the last tile, and how many of its blocks
        if (lane == 0) {
          for (int k = c; k < 3; ++k) mbar_arrive(&k_full[g & 1]);
          for (int k = max(c, 3); k < 5; ++k) mbar_arrive(&v_full[g & 1]);
        }
        __syncwarp();
        for (int t = max(0, g - 1); t <= g; ++t) {
          mbar_wait(&k_full[t & 1], (t >> 1) & 1, nullptr, 100000000ull);
          mbar_wait(&v_full[t & 1], (t >> 1) & 1, nullptr, 100000000ull);
        }
      }
    } else if (warp >= 18) {
      // ====================================================== values
      const int ct = tid - 18 * 32;
      int done = 0;
      bool ok = true;
      for (int sg = 0; ok; ++sg) {
        if (!bar_warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
        const volatile XStretch& seg = *seg_at(sg);
        if (!(seg.flags & XST_SOME)) break;
        const int k0 = seg.k0, n = seg.k1 - k0, lo = seg.lo, hi = seg.hi, all_lo = seg.all_lo, all_hi = seg.all_hi;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int g = done + j, t0 = (k0 + j) * XKT;
#pragma unroll 1
          for (int half = 0; half < 2 && ok; ++half) {
            const int slot = (5 * g + 3 + half) & (XRING - 1);
            if (half == 0) ok = bar_warp_wait(&v_full[g & 1], (g >> 1) & 1, abort_flag);
            if (!ok) break;
            if (t0 + XKT <= all_hi && t0 >= all_lo) continue;
            uint8_t* blk = sm + LY::RING + slot * XBLK;
            bool odd = false;
#pragma unroll 4
            for (int c = ct; c < XBLK / 16; c += 64) {   // 16-byte pieces: [2][64 keys][8]
              const int key = t0 + 64 * half + (c >> 3 & 63);
              uint4* at = reinterpret_cast<uint4*>(blk) + c;
              uint4 w = *at;
              if (key >= hi || key < lo) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (drop_nonfinite<T>(w.x) | drop_nonfinite<T>(w.y) | drop_nonfinite<T>(w.z) | drop_nonfinite<T>(w.w)) {
                *at = w;
                odd = true;
              }
            }
            if (odd) *odd_seen = 1;
          }
          if (!ok) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[g & 1]);
        }
        done += n;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&a.pv.state[PST_ERR], DEVERR_TIMEOUT);
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
template <typename T>
static cudaError_t prepare_t() {
  // reg_inc draws on the registers that the block was launched with: fewer
  // would make it wait for ever
  cudaFuncAttributes fa;
  const cudaError_t e = cudaFuncGetAttributes(&fa, latent_expanded_kernel<T>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * XTHREADS < 32 * (16 * kXSoftmaxRegs + 4 * kXOtherRegs)) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(latent_expanded_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, XLayout::ALLOC);
}

cudaError_t prepare_latent_expanded() {
  const cudaError_t e = prepare_t<__half>();
  return e == cudaSuccess ? prepare_t<__nv_bfloat16>() : e;
}

template <typename T>
static cudaError_t expanded_t(const ExpandedAttn& xa, const CUtensorMap& tmK, const CUtensorMap& tmR,
                              const CUtensorMap& tmV, int blocks, cudaStream_t st) {
  return launch_pdl(latent_expanded_kernel<T>, dim3(blocks), dim3(XTHREADS), XLayout::ALLOC, st, tmK, tmR, tmV, xa);
}

cudaError_t launch_latent_expanded(const ExpandedAttn& xa, const CUtensorMap& tmK, const CUtensorMap& tmR,
                                   const CUtensorMap& tmV, bool f16, int sms, cudaStream_t st) {
  const int blocks = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  const cudaError_t e = f16 ? expanded_t<__half>(xa, tmK, tmR, tmV, blocks, st)
                            : expanded_t<__nv_bfloat16>(xa, tmK, tmR, tmV, blocks, st);
  return e == cudaSuccess ? launch_latent_join(xa.a, xa.o, XTR, XTR, f16, blocks, st) : e;
}

}  // namespace kvring_dev
