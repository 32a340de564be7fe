// paged_attend_tiles: attention of many query rows over a paged FP8 cache, on
// the tcgen05 tensor cores.
//
// The same sums as the row kernel's (y_t with log2 s_v as an offset, weights
// of the V codes, l divided by s_v), over tiles:
//   S = Q K^T      kind::f16, Q fp16 (rotated, power-of-two row scale), K codes widened
//   P = 2^(y - m + 6), fp16, stored in tensor memory over the S it came from
//   O += P V       kind::f16, A = P from tensor memory, V codes widened
// fp16 holds every e4m3 code exactly, so the products add no rounding to the
// cache's own; e4m3 operands would, Q and P having 3 bits of fraction there.
// An fp16 query carries more bits than one fp16 number holds after the
// rotation, and its output shows them: for that type Q = Q_hi + Q_lo, two
// products into one S.  The weights are one fp16 number for either type (half a
// step: 2^-11, as the fp16 output's own): a low part would be a second PV and
// room for it in a tensor memory that is full.
//
// What bounds it: the tensor pipe (128 x 128 x 16 fp16 in about 64 cycles),
// beside which the softmax and the widening have to run.  A block works on two
// tiles of 128 query rows over the same keys, so that each K and V tile is
// loaded and widened once for 256 rows and the tensor cores work on one tile
// while the softmax of the other runs.  Tensor memory is full: S (then P) and O
// of both.  S is 128 keys wide in one product: with two buffers of 64 keys QK
// could run ahead of the softmax, but a 128 x 64 x 16 product from shared memory
// takes 58 cycles, hardly less than a 128 x 128 x 16 one.
// Measured: 512 tokens over 65,000, 32 query heads on 8 key heads: 466 us
// (1.17 PFLOP/s, 63% of a library product); three prompts of 1,731 to 3,644
// tokens 313 us (0.65 PFLOP/s).  128 keys of 256 rows take some 4,000 cycles: the
// products 2,200, the chain of one query tile (softmax 2,000, its two products
// 1,100, hand-overs) the rest, beside widening that is nearly as long; without any
// exponential, or any conversion, the kernel was no more than 2% faster.  A piece
// of an item costs some 12,000 cycles beside its tiles (queries 6,500, the last
// product and the results 5,000), and its phases' code does not stay in the
// instruction caches (0.9 of 9 stalled warps per issue in the prompts, none worth
// naming in the long chunk).
//
// Warp roles (640 threads, registers moved from the last group to the softmax):
//   warps 0-15       softmax: of query tile t and half p of its keys, warps
//                    8 p + 4 t .. + 3, one row per thread: two warps share a row.
//                    They also load and rotate the rows' queries and write the output
//   warp 16          MMA issue
//   warp 17          the line of work: the stretches of items for the others,
//                    per tile the page ids and scales, and TMA of the codes
//   warps 18, 19     K and V codes widened to fp16, shared memory to shared memory
// QK of the next tile overwrites the P that PV of this one reads, with another
// accumulator: products of different accumulators have no documented order, so
// it is issued once that PV has completed.
#include "paged_exact.cuh"
#include "paged_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int TM_ROWS = 128;                 // rows of one MMA
constexpr int TTR = kTilesRows;              // rows of an item: two query tiles
static_assert(TTR == 2 * TM_ROWS);
constexpr int TTHREADS = 640;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;   // per thread: 16 warps and 4
constexpr int TMETA = 3;                     // stages of page ids and scales
constexpr float kRaise = 8.0f;               // a row's maximum is raised when a tile exceeds it by 2^8 ...
constexpr float kTop = 6.0f;                 // ... and starts its weights at 2^6, so they stay below 2^14 in fp16

// What a block does of one item: its key tiles [k0, k1).  Some row sees keys
// lo .. hi - 1, all rows see all_lo .. all_hi - 1.
struct Stretch {
  int b, h, tile, s0, n, len, lo, hi, all_lo, all_hi, k0, k1, flags;
  int far_apart;                             // its pages' V scales (written with the last tile's)
  int pad[2];
};
enum : int { STRETCH_SOME = 1, STRETCH_WHOLE = 2, STRETCH_HEAD = 4 };   // else: the end; the whole item; its beginning

template <int D, typename T>
struct TilesLayout {
  static constexpr int NQ = std::is_same_v<T, __half> ? 2 : 1;   // fp16 parts of a query
  static constexpr int KT = NQ == 2 ? 64 : 128;                  // keys per K and V tile
  static constexpr int QB = TM_ROWS * D * 2;                     // one part of one query tile
  static constexpr int KB = KT * D * 2;                          // one widened K or V tile
  static constexpr int Q = 0;                                    // [2 tiles][NQ]
  static constexpr int KH = Q + 2 * NQ * QB;                     // [2]
  static constexpr int VH = KH + 2 * KB;                         // [2]
  static constexpr int RAW = VH + 2 * KB;                        // K codes, V codes of one tile
  static constexpr int META = RAW + 2 * KT * D;                  // [TMETA][KT / 16] {s_k, log2 s_v, 1 / s_v, -}
  static constexpr int SLOT = META + TMETA * (KT / 16) * 16;     // [2 halves][256] a row's logit factor; maxima; sums
  static constexpr int SUMS = SLOT + 1024;                       // (at first) sums over the items, behind the warps'
  static constexpr int SEG = SLOT + 2 * TTR * 4;                 // [2] Stretch
  static constexpr int BAR = SEG + 2 * (int)sizeof(Stretch);
  static constexpr int NBAR = 2 + 2 + 2 + TMETA + 4 + 4 + 2 + 4 + 4 + 1 + 16 + 8;
  static constexpr int MISC = BAR + NBAR * 8;
  static constexpr int ALLOC = MISC + 16;                        // the block's shared memory starts 1024-byte aligned
  static_assert(ALLOC <= 232448, "shared memory of a block");
  static_assert(KH >= (kPagedMaxSeqs + 1) * 8, "the prefix sums lie in the query tiles at first");
};

// byte offset of 16-byte chunk c of code row r as TMA left it (128- or 64-byte swizzle)
template <int D>
__device__ __forceinline__ int raw_chunk(int r, int c) {
  if constexpr (D == 128)
    return r * 128 + ((c ^ (r & 7)) << 4);
  else
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Whether one of the values of keys lo, lo + 2, .. < hi holds a NaN code, keys
// that every row sees left out (tiles of KT keys inside [all_lo, all_hi)).
template <int D, int KT>
__device__ __noinline__ bool nan_among(const PagedAttn& a, int b, int h, int lo, int hi, int all_lo, int all_hi) {
#pragma unroll 1
  for (int key = lo; key < hi; key += 2) {
    const int k = key / KT;
    if (k * KT >= all_lo && k * KT + KT <= all_hi) continue;
    int pg = a.pb.table[b * a.pb.table_stride + (key >> a.pv.p_shift)];
    if (pg < 0 || pg >= a.pv.n_pages) pg = 0;
    const uint4* v = reinterpret_cast<const uint4*>(
        a.pv.v_codes + (((((size_t)pg * a.pv.H + h) << a.pv.p_shift) + (key & (a.pv.P - 1))) * D));
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
      uint4 w = v[c];
      if (drop_nan_codes(w.x) | drop_nan_codes(w.y) | drop_nan_codes(w.z) | drop_nan_codes(w.w)) return true;
    }
  }
  return false;
}

template <int D, typename T>
__global__ void __launch_bounds__(TTHREADS, 1)
    paged_attend_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                              const __grid_constant__ PagedAttn a) {
  using LY = TilesLayout<D, T>;
  constexpr int KT = LY::KT, NQ = LY::NQ, NG = KT / 16;
  constexpr int SC = KT / 2;               // keys of a tile that a softmax warp looks at
  using SH = Share<TTR, KT, 2, kRowsMax, 0x7FFFFFFF>;
  constexpr uint32_t TM_S = 0, TM_O = 256;
  constexpr int kNone = -1;                // page of a group of keys that no query sees
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR);
  uint64_t* q_full = bars;                 // [2] query tile written (once per stretch)
  uint64_t* kh_full = q_full + 2;          // [2] K tile widened
  uint64_t* vh_full = kh_full + 2;         // [2] V tile widened
  uint64_t* meta_free = vh_full + 2;       // [TMETA] the tile's softmax is done
  uint64_t* s_full = meta_free + TMETA;    // [2 query tiles][2] QK done
  uint64_t* o_done = s_full + 4;           // [2][2] PV done
  uint64_t* p_full = o_done + 4;           // [2] P stored
  uint64_t* raw_full = p_full + 2;         // [2] K codes, V codes landed
  uint64_t* raw_free = raw_full + 2;       // [2] and read
  uint64_t* seg_full = raw_free + 2;       // [2] stretch written
  uint64_t* seg_free = seg_full + 2;       // [2] every role is done with it
  uint64_t* drain = seg_free + 2;          // every MMA done
  uint64_t* m_ready = drain + 1;           // [2][4 warps][2 halves] a half's maxima written
  uint64_t* both = m_ready + 16;           // [2][4] both warps of a row are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC + 4);
  volatile int* nan_seen = reinterpret_cast<volatile int*>(sm + LY::MISC + 8);   // see the K, V warps
  volatile Stretch* segs = reinterpret_cast<volatile Stretch*>(sm + LY::SEG);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 8);
      mbar_init(&kh_full[i], 2);
      mbar_init(&vh_full[i], 2);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], 2);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_free[i], 19);
    }
    for (int i = 0; i < TMETA; ++i) {
      mbar_init(&meta_free[i], 16);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&p_full[i], 8);
    for (int i = 0; i < 16; ++i) mbar_init(&m_ready[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&both[i], 2);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *nan_seen = 0;
    for (int i = 0; i < 3; ++i) reinterpret_cast<unsigned long long*>(sm + LY::SUMS)[i] = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 17 && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  // this block's stretch of the line of items
  long long* pre = reinterpret_cast<long long*>(sm + LY::Q);
  const Cut cut = SH::template prefix<TTHREADS>(a, pre, reinterpret_cast<long long*>(sm + LY::SLOT), false,
                                                reinterpret_cast<unsigned long long*>(sm + LY::SUMS), gridDim.x);
  const int H = a.pv.H, G = a.pv.G;
  const long long total = pre[a.pb.n_seqs] * H;
  long long stretch = quotient(total + gridDim.x - 1, gridDim.x);
  if (stretch < SH::kLeast) stretch = SH::kLeast;
  if (cut.pad) stretch = cut.stretch;
  const int worker = blockIdx.x;
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  Place pl;
  if (warp == 17 && u < end) pl = find_place<SH, TTR, KT>(a, pre, u, cut.pad);
  __syncthreads();                         // the prefix sums' room is the query tiles' now

  // ``done``: tiles of the line that a role has behind it; it gives the stage
  // and phase of every per-tile barrier.  Waits tell a phase only from the one
  // before it, so no barrier may complete twice before all of its waiters have
  // seen the first: a role that has nothing to do in a tile still waits, and
  // arrives where the next phase needs that it has.
  if (warp < 16) {
    // ======================================================== softmax
    reg_inc<kSoftmaxRegs>();
    const int t = (warp >> 2) & 1;
    const int par = warp >> 3;
    const int row = tid & 127;
    float* slots = reinterpret_cast<float*>(sm + LY::SLOT) + t * TM_ROWS + row;
    float *mine = slots + par * TTR, *other = slots + (par ^ 1) * TTR;
    const int pair = 4 * t + (warp & 3);   // the two warps of these rows
    uint32_t nb = 0, tiles = 0;            // phases of ``both``, and of the barriers of this query tile's key tiles
    auto meet = [&]() {                    // the other warp need not be here yet
      __syncwarp();
      if (lane == 0) mbar_arrive(&both[pair]);
      ++nb;
    };
    auto met = [&]() -> bool { return warp_wait(&both[pair], (nb - 1) & 1, abort_flag); };
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + TM_S + 128 * t + SC * par;
    const uint32_t o_at = tmem + lanes + TM_O + 128 * t;
    int done = 0;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      if (!warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
      const volatile Stretch& seg = segs[sg & 1];
      const int flags = seg.flags;
      if (!(flags & STRETCH_SOME)) break;
      const int k0 = seg.k0, n = seg.k1 - k0, len_n = seg.len - seg.n, s0 = seg.s0;
      const int rows = min(TM_ROWS, seg.n * G - seg.tile * TTR - t * TM_ROWS);   // of this query tile
      const int r0 = seg.tile * TTR + t * TM_ROWS;
      const int head0 = seg.h * G;
      const bool live = row < rows;
      const int i = live ? (r0 + row) / G : 0;
      const int hi = !live ? 0x7FFFFFFF : a.causal ? len_n + i + 1 : seg.len;
      const int lo = live && a.window > 0 ? len_n + i - a.window + 1 : 0;
      float m = -INFINITY, l = 0.0f;
      if (nb > 0 && !met()) break;                       // the other warp is done with the last stretch
      if (n > 0 && rows > 0) {
        // ------------------------------------------------------ queries
        // the pair its own 32 rows, a warp every other turn, a row by L lanes of
        // 16 channels; the turns' loads in flight together
        constexpr int L = D / 16;
        constexpr int RSTEP = 32 / L;                    // rows per turn
        constexpr int BATCH = 2;
        static_assert(32 % (2 * RSTEP * BATCH) == 0);
        const int ql = tid % L;
        const int rr0 = 32 * (warp & 3) + 16 * par + lane / L;
        float* rfs = reinterpret_cast<float*>(sm + LY::SLOT) + t * TM_ROWS;
        const RopeLane rl = rope_lane(a.pv, ql * 8);
        bool bad = false;
        // the token and head of a row, carried from one turn to the next
        const int step_i = RSTEP / G, step_g = RSTEP - step_i * G;
        int qi = (r0 + rr0) / G, qg = r0 + rr0 - qi * G;
        const T* qp = static_cast<const T*>(a.q) + (size_t)head0 * D + ql * 16;
        const int32_t* pr0 = a.q_pos + (size_t)s0 * a.pv.n_axes;
        auto step = [&](int& i2, int& g2) {
          i2 += step_i;
          g2 += step_g;
          if (g2 >= G) {
            g2 -= G;
            ++i2;
          }
        };
        // positions of a turn's rows, a turn ahead of its loads from the table
        int idx[BATCH];
        auto positions = [&](int rr, int i2, int g2) {
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            idx[k] = rope_index(rl, pr0 + (size_t)(rr + k * RSTEP < rows ? i2 : 0) * a.pv.n_axes);
            step(i2, g2);
          }
        };
        positions(rr0, qi, qg);
#pragma unroll 1
        for (int rr = rr0; rr < 32 * (warp & 3) + 16 * par + 16; rr += RSTEP * BATCH) {
          uint4 w0[BATCH], w1[BATCH];
          float2 cs[BATCH][8];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const bool on = rr + k * RSTEP < rows;       // rows past the last: zeros
            w0[k] = w1[k] = make_uint4(0, 0, 0, 0);
            if (on) {
              const uint4* src = reinterpret_cast<const uint4*>(qp + (s0 + qi) * a.q_stride + qg * D);
              w0[k] = src[0];
              w1[k] = src[1];
            }
            rope_load(a.pv, rl, pr0 + (size_t)(on ? qi : 0) * a.pv.n_axes, idx[k], cs[k], bad);
            step(qi, qg);
          }
          positions(rr + RSTEP * BATCH, qi, qg);         // (rows past the last turn's: a row's position all the same)
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const int rk = rr + k * RSTEP;
            uint32_t mb = __vmaxu2(max8_bits(w0[k]), max8_bits(w1[k]));
#pragma unroll
            for (int off = L / 2; off > 0; off >>= 1) mb = __vmaxu2(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, off));
            const int ex = query_exponent<T>(mb);
            const float down = pow2f(-ex);
            if (ql == 0) rfs[rk] = a.scale_log2 * pow2f(ex);
            float x[16];
            load8_f32<T>(w0[k], x);
            load8_f32<T>(w1[k], x + 8);
            uint8_t* dst = sm + LY::Q + t * NQ * LY::QB + (ql >> 2) * (TM_ROWS * 128) + rk * 128;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[4], v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = mul2(rope_query(x[8 * c + 2 * e], x[8 * c + 2 * e + 1], cs[k][4 * c + e]),
                                      make_float2(down, down));
                w[e] = cvt_f16x2(y.x, y.y);
                if constexpr (NQ == 2) {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                  v[e] = cvt_f16x2(y.x - f.x, y.y - f.y);
                }
              }
              uint8_t* at = dst + (((2 * ql + c) & 7) ^ (rk & 7)) * 16;
              *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
              if constexpr (NQ == 2) *reinterpret_cast<uint4*>(at + LY::QB) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
        meet();
        if (!met()) ok = false;
        const float rf = slots[0];
        meet();                                          // (both have read it: waited for before the first maxima)
        // ------------------------------------------------------ key tiles
        // tiles below j_lo and from j_hi on hold keys that some row of the warp does not see
        const int past = hi - k0 * KT - (par + 1) * SC, before = lo - k0 * KT - par * SC;
        const int j_hi = __reduce_min_sync(0xFFFFFFFFu, past >= 0 ? past / KT + 1 : 0);
        const int j_lo = __reduce_max_sync(0xFFFFFFFFu, before > 0 ? (before + KT - 1) / KT : 0);
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j, ++tiles) {
          const int g = done + j;
          if (!warp_wait(&s_full[2 * t + (g & 1)], (g >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int stage = g % TMETA;
          const float4* meta = reinterpret_cast<const float4*>(sm + LY::META) + stage * NG + par * (NG / 2);
          uint32_t xr[SC];
          if constexpr (SC == 64) tmem_ld_32x32b_x64(s_at, xr);
          else tmem_ld_32x32b_x32(s_at, xr);
          if (j >= j_hi || j < j_lo) {
            const int key0 = (k0 + j) * KT + par * SC;
#pragma unroll
            for (int k = 0; k < SC; ++k)
              if (key0 + k >= hi || key0 + k < lo) xr[k] = 0xFF800000u;   // -inf
          }
          const float* s = reinterpret_cast<const float*>(xr);
          // a factor is never 0, so that a masked score stays -inf
          float my = -INFINITY;
#pragma unroll
          for (int q = 0; q < SC / 16; ++q) {
            const float2 mt = *reinterpret_cast<const float2*>(meta + q);
            const float* v = s + 16 * q;
            const float a0 = max3f(v[0], v[1], v[2]), a1 = max3f(v[3], v[4], v[5]), a2 = max3f(v[6], v[7], v[8]);
            const float a3 = max3f(v[9], v[10], v[11]), a4 = max3f(v[12], v[13], fmaxf(v[14], v[15]));
            my = fmaxf(my, fmaf(max3f(max3f(a0, a1, a2), a3, a4), fmaxf(rf * mt.x, 0x1p-100f), mt.y));
          }
          // the row's maximum: the other half's keys are the other warp's.  Both
          // see the same numbers and do the same.
          if (j == 0 && !met()) ok = false;
          *mine = my;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_ready[2 * pair + par]);
          if (!warp_wait(&m_ready[2 * pair + (par ^ 1)], tiles & 1, abort_flag)) ok = false;
          const float mm = fmaxf(my, *other);
          if (__any_sync(0xFFFFFFFFu, mm > m + kRaise)) {
            // rare after a row's first keys: what was summed with the old
            // maximum is brought to the new one
            const float mn = mm > m + kRaise ? mm : m;
            const float al = mn > m ? ex2f(m - mn) : 1.0f;     // 0 for the row's first keys
            m = mn;
            l *= al;
            if (j > 0) {
              // QK of this tile was issued after the PV before it, so that one is done
              if (!warp_wait(&o_done[2 * t + ((g - 1) & 1)], ((g - 1) >> 1) & 1, abort_flag)) ok = false;
              tc_fence_after();
#pragma unroll 1
              for (int k = par * (D / 2); k < (par + 1) * (D / 2); k += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(o_at + k, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st_32x32b_x16(o_at + k, o);
              }
            }
          }
          const float sub = m == -INFINITY ? 0.0f : kTop - m;
#pragma unroll
          for (int c = 0; c < SC / 32; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int q = 2 * c + e;
              const float4 mt = meta[q];
              const float f = fmaxf(rf * mt.x, 0x1p-100f), ad = mt.y + sub;
              float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float2 y = fma2(make_float2(s[16 * q + 2 * k], s[16 * q + 2 * k + 1]), make_float2(f, f),
                                make_float2(ad, ad));
                y.x = ex2f(y.x);
                y.y = ex2f(y.y);
                part = add2(part, y);
                p[8 * e + k] = cvt_f16x2(y.x, y.y);
              }
              l = fmaf(part.x + part.y, mt.z, l);
            }
            tmem_st_32x32b_x16(s_at + 16 * c, p);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_full[t]);
            mbar_arrive(&meta_free[stage]);
          }
        }
      } else {
        for (int j = 0; ok && j < n; ++j) {
          const int g = done + j;
          ok = warp_wait(&s_full[2 * t + (g & 1)], (g >> 1) & 1, abort_flag);
          if (lane == 0) {
            mbar_arrive(&p_full[t]);
            mbar_arrive(&meta_free[g % TMETA]);
          }
        }
      }
      done += n;
      if (ok && n > 0) ok = warp_wait(&o_done[2 * t + ((done - 1) & 1)], ((done - 1) >> 1) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (*nan_seen && n > 0 && live &&
          nan_among<D, KT>(a, seg.b, seg.h, max(max(lo, seg.lo), k0 * KT) + par, min(min(hi, seg.hi), (k0 + n) * KT), seg.all_lo,
                           seg.all_hi))
        l = __int_as_float(0x7FFFFFFF);                  // the row sees one of the values left out
      if (n > 0 && rows > 0) {
        // the row's sum: both halves
        *mine = l;
        meet();
        if (!met()) break;
        l = slots[0] + slots[TTR];
      }
      // -------------------------------------------------------- results
      // Half of the channels per warp.  A thread has a row, memory wants rows side
      // by side in a warp: through half of the warp's rows of the query tile,
      // which every MMA is done with.
      if (n > 0 && seg.far_apart) {
        // half of the pair's rows each
        for (int r = 32 * (warp & 3) + 16 * par; r < min(rows, 32 * (warp & 3) + 16 * par + 16); ++r) {
          const int i2 = (r0 + r) / G;
          const size_t at = (size_t)(2 * worker + (flags & STRETCH_HEAD ? 1 : 0)) * TTR + t * TM_ROWS + r;
          T* dst = static_cast<T*>(a.out) + (s0 + i2) * a.out_stride + (size_t)(head0 + r0 + r - i2 * G) * D;
          exact_row<D, T>(a, seg.b, s0, seg.n, seg.len, seg.h, r0 + r, k0 * KT, (k0 + n) * KT,
                          flags & STRETCH_WHOLE ? dst : nullptr, a.tiles.o + at * D, a.tiles.ml + at, kTop);
        }
      } else if (rows > 0) {
        const bool whole = flags & STRETCH_WHOLE;
        const size_t at_row = (size_t)(2 * worker + (flags & STRETCH_HEAD ? 1 : 0)) * TTR + t * TM_ROWS + row;
        constexpr int HC = D / 16;                       // 16-byte chunks of half a row of the tile
        uint8_t* own = sm + LY::Q + t * NQ * LY::QB + 32 * (warp & 3) * 128 + (D == 128 ? par * (TM_ROWS * 128) : 0);
        const int c0 = D == 128 ? 0 : par * HC;          // the warp's chunks of the 128-byte row
        auto put = [&](int c, uint4 v) {                 // chunk c of the thread's row
          *reinterpret_cast<uint4*>(own + lane * 128 + (((c0 + c) ^ (lane & 7)) << 4)) = v;
        };
        auto flush = [&](void* dst) {                    // the chunks of every row to the row's dst
          __syncwarp();
#pragma unroll
          for (int i = 0; i < HC; ++i) {
            const int rr = i * (32 / HC) + lane / HC, c = lane % HC;
            const unsigned long long p = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(dst), rr);
            const uint4 v = *reinterpret_cast<const uint4*>(own + rr * 128 + (((c0 + c) ^ (rr & 7)) << 4));
            if (p) reinterpret_cast<uint4*>(p)[c] = v;
          }
          __syncwarp();
        };
        if (whole) {
          const float inv = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            if (n > 0) {
              tmem_ld_32x32b_x32(o_at + par * (D / 2) + c, o);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<T>(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
              put(c / 8 + k, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          T* dst = static_cast<T*>(a.out) + (s0 + i) * a.out_stride +
                   (size_t)(head0 + (live ? r0 + row - i * G : 0)) * D + par * (D / 2);
          flush(live ? dst : nullptr);
        } else {
          if (live && par == 0) a.tiles.ml[at_row] = make_float2(m, l);
          if (n > 0) {
            // fp32: half of the warp's channels at a time
#pragma unroll 1
            for (int h4 = par * (D / 2); h4 < (par + 1) * (D / 2); h4 += D / 4) {
              uint32_t o[D / 4];
              if constexpr (D == 128) tmem_ld_32x32b_x32(o_at + h4, o);
              else tmem_ld_32x32b_x16(o_at + h4, o);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) put(k, make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
              flush(live ? a.tiles.o + at_row * D + h4 : nullptr);
            }
          }
        }
      }
      tc_fence_before();
      // sums read, rows of the query tile free: waited for before the next queries
      meet();
      if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
    }
  } else {
    reg_dec<kOtherRegs>();
    if (warp == 16) {
      // ====================================================== MMA issue
      if (lane == 0) {
        constexpr uint32_t idesc_qk = make_idesc(0, 0, 0, 0, TM_ROWS, KT);
        constexpr uint32_t idesc_pv = make_idesc(0, 0, 0, 1, TM_ROWS, D);
        const uint32_t q0 = smem_u32(sm + LY::Q), kh0 = smem_u32(sm + LY::KH), vh0 = smem_u32(sm + LY::VH);
        uint32_t nq0 = 0, nq1 = 0;                       // stretches of either query tile so far
        int done = 0;
        // 64 channels (a column block of 128-byte rows) per turn of the loop
        auto qk = [&](int t, int g) {
          const uint32_t q = q0 + t * NQ * LY::QB, kh = kh0 + (g & 1) * LY::KB;
#pragma unroll 1
          for (int c = 0; c < NQ * (D / 64); ++c) {
            const int block = c & (D / 64 - 1), part = c / (D / 64);
            mma4_f16_ss(tmem + TM_S + 128 * t, make_sdesc_sw128(q + part * LY::QB + block * (TM_ROWS * 128), 16, 1024),
                        make_sdesc_sw128(kh + block * (KT * 128), 16, 1024), idesc_qk, c);
          }
        };
        // both halves of the tile's keys, each half's P over its S
        auto pv = [&](int t, int g, uint32_t accumulate) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint64_t b = make_sdesc_sw128(vh0 + (g & 1) * LY::KB + half * SC * 128, KT * 128, 1024);
            const uint32_t p = tmem + TM_S + 128 * t + half * SC;
            if constexpr (SC == 64) mma4_f16_ts(tmem + TM_O + 128 * t, p, b, idesc_pv, accumulate | half);
            else mma2_f16_ts(tmem + TM_O + 128 * t, p, b, idesc_pv, accumulate | half);
          }
        };
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
          if (!mbar_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
          const volatile Stretch& seg = segs[sg & 1];
          if (!(seg.flags & STRETCH_SOME)) break;
          const int n = seg.k1 - seg.k0;
          const bool two = seg.n * G - seg.tile * TTR > TM_ROWS;   // the second query tile has rows
          if (n > 0) {
            ok = mbar_wait(&kh_full[done & 1], (done >> 1) & 1, abort_flag) && mbar_wait(&q_full[0], nq0++ & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            qk(0, done);
            mma_commit(&s_full[done & 1]);
            if (two) {
              ok = mbar_wait(&q_full[1], nq1++ & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              qk(1, done);
            }
            mma_commit(&s_full[2 + (done & 1)]);
          }
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j) {
            const int g = done + j;
            ok = mbar_wait(&vh_full[g & 1], (g >> 1) & 1, abort_flag) &&
                 (j + 1 >= n || mbar_wait(&kh_full[(g + 1) & 1], ((g + 1) >> 1) & 1, abort_flag));
#pragma unroll 1
            for (int t = 0; t < 2 && ok; ++t) {
              const bool on = t == 0 || two;
              ok = mbar_wait(&p_full[t], g & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              if (on) pv(t, g, j > 0);
              mma_commit(&o_done[2 * t + (g & 1)]);
              if (j + 1 < n) {
                if (on) {
                  ok = mbar_wait(&o_done[2 * t + (g & 1)], (g >> 1) & 1, abort_flag);
                  if (!ok) break;
                  tc_fence_after();
                  qk(t, g + 1);
                }
                mma_commit(&s_full[2 * t + ((g + 1) & 1)]);
              }
            }
          }
          if (!ok) break;
          done += n;
          mbar_arrive(&seg_free[sg & 1]);
        }
        // every MMA issued so far is done before the block releases its tensor memory
        mma_commit(drain);
        mbar_wait(drain, 0, nullptr, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 17) {
      // ====================================================== the line of work
      PieceRec rec = {};
      const int rows = a.pv.P < 32 ? a.pv.P : 32;
      // Codes leave the L2 first: a sequence longer than it pushes nothing else
      // out (65,000 cached tokens, two builds that differed in this alone: 490 us
      // without the hint, 474 with it)
      const uint64_t once = l2_evict_first();
      int done = 0, sg = 0, issued = 0;                  // tiles, stretches; copies (K, V, K, ...)
      bool ok = true;
      for (bool more = u < end; ok; ++sg) {
        if (sg >= 2 && !warp_wait(&seg_free[sg & 1], ((sg - 2) >> 1) & 1, abort_flag)) break;
        int k0 = 0, k1 = 0;
        long long item_end = 0;
        if (more) {
          item_end = pl.at + pl.units;
          const int n = pl.t.t1 - pl.t.t0;
          k0 = pl.t.t0 + (int)max(0ll, min((long long)n, u - pl.at - 2));
          k1 = pl.t.t0 + (int)max(0ll, min((long long)n, min(end, item_end) - pl.at - 2));
        }
        if (lane == 0) {
          volatile Stretch& seg = segs[sg & 1];
          if (more) {
            const bool head = u == pl.at;
            seg.b = pl.b;
            seg.h = pl.h;
            seg.tile = pl.tile;
            seg.s0 = pl.s.s0;
            seg.n = pl.s.n;
            seg.len = pl.s.len;
            seg.lo = pl.t.lo;
            seg.hi = pl.t.hi;
            const int i0 = pl.tile * TTR / G, i1 = min(pl.s.n - 1, (pl.tile * TTR + TTR - 1) / G);
            seg.all_hi = a.causal ? pl.s.len - pl.s.n + i0 + 1 : pl.s.len;
            seg.all_lo = a.window > 0 ? pl.s.len - pl.s.n + i1 - a.window + 1 : 0;
            seg.far_apart = 0;
            seg.k0 = k0;
            seg.k1 = k1;
            seg.flags = STRETCH_SOME | (head ? STRETCH_HEAD : 0) | (head && end >= item_end ? STRETCH_WHOLE : 0);
          } else {
            seg.flags = 0;
          }
          mbar_arrive(&seg_full[sg & 1]);
        }
        __syncwarp();
        if (!more) break;
        // page ids and scales of its tiles: lane i the keys 16 i .. 16 i + 15,
        // which lie in one page.  Pages of zero values take a V scale near by.
        const int32_t* tab = a.pb.table + pl.b * a.pb.table_stride;
        float near = 0.0f;
        ScaleSpan span;
        // (Loads run a tile ahead: TMA of the next tile waits for nothing else than its stage.)
        auto page = [&](int k) -> int {
          const int key = k * KT + lane * 16;
          return lane < NG && k < k1 && key < pl.t.hi && key + 16 > pl.t.lo ? tab[key >> a.pv.p_shift] : -0x7FFFFFFF;
        };
        auto known = [&](int pg) -> int {                // a page that can be read
          if (pg == -0x7FFFFFFF) return kNone;
          if (pg < 0 || pg >= a.pv.n_pages) {
            atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
            return 0;
          }
          return pg;
        };
        auto scale = [&](const float* scales, int pg) {
          return pg != kNone ? scales[(size_t)pg * H + pl.h] : 0.0f;
        };
        auto top = [](float v) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
          return v;
        };
        int pg = kNone;
        float sk = 0.0f, sv = 0.0f;
        if (k0 < k1) {
          pg = known(page(k0));
          sk = scale(a.pv.k_scale, pg);
          sv = scale(a.pv.v_scale, pg);
        }
        for (int k = k0; k < k1; ++k) {
          const int g = done + k - k0;
          const int next = page(k + 1);
          span.add(sv);
          float mx = top(sv);
          if (mx == 0.0f && near == 0.0f) {
            for (int s = k + 1; mx == 0.0f && s < k1; ++s) mx = top(scale(a.pv.v_scale, known(page(s))));
            if (mx == 0.0f) mx = 1.0f;
          }
          if (mx > 0.0f) near = mx;
          if (g >= TMETA && !warp_wait(&meta_free[g % TMETA], ((g - TMETA) / TMETA) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (k + 1 == k1) {
            const bool far = span.far_apart();
            if (lane == 0) segs[sg & 1].far_apart = far;
          }
          if (lane < NG) {
            const float v = sv > 0.0f ? sv : near;
            reinterpret_cast<float4*>(sm + LY::META)[(g % TMETA) * NG + lane] =
                make_float4(sk, __log2f(v), 1.0f / v, 0.0f);
          }
          __syncwarp();
          // the codes, lane i a box of the tile: 32 rows of a page (16 where a
          // page has no more)
          const int box_pg = rows == 16 ? pg : max(__shfl_sync(0xFFFFFFFFu, pg, (2 * lane) & 31),
                                                   __shfl_sync(0xFFFFFFFFu, pg, (2 * lane + 1) & 31));
          const bool on = lane < KT / rows && box_pg != kNone;
          const int key = k * KT + lane * rows;
          const int y = (int)(a.pv.row0 + (((long long)box_pg * H + pl.h) << a.pv.p_shift)) + (key & (a.pv.P - 1));
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, on)) * rows * D;
#pragma unroll 1
          for (int v = 0; v < 2; ++v) {
            if (g >= 1 && !warp_wait(&raw_free[v], (g - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[v], bytes);
            __syncwarp();
            if (on) tma_load_2d_hint(sm + LY::RAW + v * KT * D + lane * rows * D, v ? &tmV : &tmK, &raw_full[v], 0, y, once);
            issued = 2 * g + v + 1;
            if (v == 0) {
              pg = known(next);
              sk = scale(a.pv.k_scale, pg);
              sv = scale(a.pv.v_scale, pg);
            }
          }
          if (!ok) break;
        }
        done += k1 - k0;
        if (u == pl.at && end < item_end)
          rec = {min(pl.s.n * G - pl.tile * TTR, TTR), (int)quotient(item_end - 1, stretch), pl.h, pl.s.s0, pl.tile * TTR};
        u = min(end, item_end);
        more = u < end && next_place<SH, TTR, KT>(a, pl, cut.pad);
      }
      if (lane == 0) a.tiles.rec[worker] = rec;
      // after an abort: copies still in flight land in this block's shared memory
      if (*abort_flag && issued > 0) {
        mbar_wait(&raw_full[0], ((issued - 1) >> 1) & 1, nullptr, 100000000ull);
        if (issued > 1) mbar_wait(&raw_full[1], ((issued - 2) >> 1) & 1, nullptr, 100000000ull);
      }
    } else {
      // ====================================================== K, V
      const int ct = tid - 18 * 32;
      constexpr int CH = D / 16;                         // 16-byte code chunks of a row
      constexpr int NT = KT * CH / 64;                   // chunks of K, and of V, per thread
      constexpr int STEP = 64 / CH;                      // rows per round of the 64 threads
      const int sl0 = CH == 8 ? ct & 7 : 8 * (ct >> 5) + (ct & 7);
      const int ch = (ct >> 3) & (CH - 1);
      int done = 0;
      bool ok = true;
      for (int sg = 0; ok; ++sg) {
        if (!warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
        const volatile Stretch& seg = segs[sg & 1];
        if (!(seg.flags & STRETCH_SOME)) break;
        const int k0 = seg.k0, n = seg.k1 - k0, lo = seg.lo, hi = seg.hi, all_lo = seg.all_lo, all_hi = seg.all_hi;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int g = done + j;
          const int buf = g & 1;
#pragma unroll 1
          for (int v = 0; v < 2; ++v) {                    // K, then V
            if (!warp_wait(&raw_full[v], g & 1, abort_flag)) {
              ok = false;
              break;
            }
            uint64_t* free = (v ? o_done : s_full) + buf;  // both query tiles are done with the buffer
            if (g >= 2 && (!warp_wait(free, ((g - 2) >> 1) & 1, abort_flag) ||
                           !warp_wait(free + 2, ((g - 2) >> 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            uint8_t* src = sm + LY::RAW + v * KT * D;
            uint8_t* dst = sm + (v ? LY::VH : LY::KH) + buf * LY::KB + (ch >> 2) * (KT * 128);
            const int cc = (2 * ch) & 7;
            const int key0 = (k0 + j) * KT;
            const bool mixed = v && (key0 + KT > all_hi || key0 < all_lo);
            if (mixed) {
              // Values that no query sees become zeros, whatever their page
              // holds; their scores are masked.  A NaN that some rows see and
              // others do not must not meet the latter's zero weights: it is
              // left out, and the sums of the rows that see it get it.  (Each
              // thread looks at the chunks that it widens below.)
#pragma unroll 1
              for (int i0 = 0; i0 < NT; i0 += 4) {
                uint4 w[4];
#pragma unroll
                for (int it = 0; it < 4; ++it)
                  w[it] = *reinterpret_cast<const uint4*>(src + raw_chunk<D>((i0 + it) * STEP + sl0, ch));
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                  const int sl = (i0 + it) * STEP + sl0, key = key0 + sl;
                  uint4* at = reinterpret_cast<uint4*>(src + raw_chunk<D>(sl, ch));
                  if (key >= hi || key < lo) {
                    *at = make_uint4(0, 0, 0, 0);
                  } else if (drop_nan_codes(w[it].x) | drop_nan_codes(w[it].y) | drop_nan_codes(w[it].z) |
                             drop_nan_codes(w[it].w)) {
                    *at = w[it];
                    *nan_seen = 1;
                  }
                }
              }
              fence_proxy_async_smem();                    // before the next codes' TMA
            }
            constexpr int BATCH = NT < 4 ? NT : 4;
#pragma unroll 1
            for (int i0 = 0; i0 < NT; i0 += BATCH) {
              uint4 reg[BATCH];
#pragma unroll
              for (int it = 0; it < BATCH; ++it) {
                const int sl = (i0 + it) * STEP + sl0;
                reg[it] = *reinterpret_cast<const uint4*>(src + raw_chunk<D>(sl, ch));
              }
#pragma unroll
              for (int it = 0; it < BATCH; ++it) {
                const int sl = (i0 + it) * STEP + sl0;
                uint32_t w[8];
                const uint32_t c[4] = {reg[it].x, reg[it].y, reg[it].z, reg[it].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  w[2 * e] = cvt_e4m3x2_to_f16x2((uint16_t)(c[e] & 0xFFFFu));
                  w[2 * e + 1] = cvt_e4m3x2_to_f16x2((uint16_t)(c[e] >> 16));
                }
                uint8_t* at = dst + sl * 128;
                *reinterpret_cast<uint4*>(at + ((cc ^ (sl & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(at + (((cc + 1) ^ (sl & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
            // The codes are given back only here: an arrival waits for no load in
            // flight, so the next codes' TMA could overwrite what a load issued
            // before it has not fetched yet.  The stores needed their values, and
            // the fence orders this proxy's reads before the copy's writes.
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&raw_free[v]);
              mbar_arrive((v ? vh_full : kh_full) + buf);
            }
          }
        }
        done += n;
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
template <int D, typename T>
static cudaError_t prepare_t() {
  // reg_inc draws on the registers that the block was launched with: fewer
  // would make it wait for ever
  cudaFuncAttributes fa;
  const cudaError_t e = cudaFuncGetAttributes(&fa, paged_attend_tiles_kernel<D, T>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * TTHREADS < 32 * (16 * kSoftmaxRegs + 4 * kOtherRegs)) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_attend_tiles_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              TilesLayout<D, T>::ALLOC);
}

cudaError_t prepare_paged_tiles(int D) {
  cudaError_t e = D == 128 ? prepare_t<128, __half>() : prepare_t<64, __half>();
  if (e == cudaSuccess) e = D == 128 ? prepare_t<128, __nv_bfloat16>() : prepare_t<64, __nv_bfloat16>();
  return e;
}

template <int D, typename T>
static cudaError_t tiles_t(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, int blocks,
                           cudaStream_t st) {
  return launch_pdl(paged_attend_tiles_kernel<D, T>, dim3(blocks), dim3(TTHREADS), TilesLayout<D, T>::ALLOC, st, tmK,
                    tmV, a);
}

cudaError_t launch_paged_tiles(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                               cudaStream_t st) {
  if (a.pv.D == 64)
    return f16 ? tiles_t<64, __half>(a, tmK, tmV, blocks, st) : tiles_t<64, __nv_bfloat16>(a, tmK, tmV, blocks, st);
  return f16 ? tiles_t<128, __half>(a, tmK, tmV, blocks, st) : tiles_t<128, __nv_bfloat16>(a, tmK, tmV, blocks, st);
}

}  // namespace kvring_dev
