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
// products into one S.
//
// What bounds it: the tensor pipe (128 x 128 x 16 fp16 in about 64 cycles),
// beside which the softmax and the widening have to run.  A block works on two
// tiles of 128 query rows over the same keys, so that each K and V tile is
// loaded and widened once for 256 rows and the tensor cores work on one tile
// while the softmax of the other runs.  S goes in steps of 64 keys through two
// buffers per query tile, so that QK of a step runs while the softmax of the
// one before it does (with one buffer of 128 keys, every tile was a chain of QK,
// softmax and PV: 577 us for 512 tokens over 65,512 against XXX).  Tensor
// memory is full: two S (then P) buffers and O of both query tiles.
//
// Warp roles (512 threads, registers moved from the last two groups to the softmax):
//   warps 0-3, 4-7   softmax of query tile 0, 1: one row per thread.  They also
//                    load and rotate the rows' queries and write the output
//   warps 8-11       K and V codes widened to fp16, shared memory to shared memory
//   warps 12, 15     MMA issue for query tile 0, 1
//   warp 13          the line of work: the stretches of items for the others,
//                    and per tile the page ids and scales, up to TMETA tiles ahead
//   warp 14          TMA: the codes of a tile, page by page
// MMAs of one thread run in the order they are issued: QK may overwrite the P
// that the PV before it reads.  A query tile has an issuing thread of its own,
// since a wait costs a thread about as much as an MMA takes.
#include "paged_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int TM_ROWS = 128;                 // rows of one MMA
constexpr int TTR = kTilesRows;              // rows of an item: two query tiles
static_assert(TTR == 2 * TM_ROWS);
constexpr int TTHREADS = 512;
constexpr int STEP_KEYS = 64;                // keys of one S buffer
constexpr int TMETA = 8;                     // stages of page ids and scales
constexpr float kRaise = 8.0f;               // a row's maximum is raised when a tile exceeds it by 2^8 ...
constexpr float kTop = 6.0f;                 // ... and starts its weights at 2^6, so they stay below 2^14 in fp16

// What a block does of one item: its key tiles [k0, k1).
struct Stretch {
  int b, h, tile, s0, n, len, lo, hi, k0, k1, flags, pad;
};
enum : int { STRETCH_SOME = 1, STRETCH_WHOLE = 2, STRETCH_HEAD = 4 };   // else: the end; the whole item; its beginning

template <int D, typename T>
struct TilesLayout {
  static constexpr int NQ = std::is_same_v<T, __half> ? 2 : 1;   // fp16 parts of a query
  static constexpr int KT = NQ == 2 ? 64 : 128;                  // keys per K and V tile
  static constexpr int SPT = KT / STEP_KEYS;                     // steps of S per tile
  static constexpr int QB = TM_ROWS * D * 2;                     // one part of one query tile
  static constexpr int KB = KT * D * 2;                          // one widened K or V tile
  static constexpr int Q = 0;                                    // [2 tiles][NQ]
  static constexpr int KH = Q + 2 * NQ * QB;                     // [2]
  static constexpr int VH = KH + 2 * KB;                         // [2]
  static constexpr int RAW = VH + 2 * KB;                        // K codes, V codes of one tile
  static constexpr int META = RAW + 2 * KT * D;                  // [TMETA][KT / 16] {s_k, log2 s_v, 1 / s_v, page}
  static constexpr int RF = META + TMETA * (KT / 16) * 16;       // [256] logit factor of a row
  static constexpr int SEG = RF + TTR * 4;                       // [2] Stretch
  static constexpr int BAR = SEG + 2 * (int)sizeof(Stretch);
  static constexpr int NBAR = 2 + 2 + 2 + 2 * TMETA + 8 + 8 + 4 + 4 + 4 + 2;
  static constexpr int SUMS = BAR + NBAR * 8;
  static constexpr int MISC = SUMS + 16 * 8;
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

template <int D, typename T>
__global__ void __launch_bounds__(TTHREADS, 1)
    paged_attend_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                              const __grid_constant__ PagedAttn a) {
  using LY = TilesLayout<D, T>;
  constexpr int KT = LY::KT, NQ = LY::NQ, NG = KT / 16, SPT = LY::SPT;
  using SH = Share<TTR, KT, 2, kRowsMax<T>, 0x7FFFFFFF>;
  constexpr uint32_t TM_S = 0, TM_O = 256;
  constexpr int kNone = -1;                // page of a group of keys that no query sees
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR);
  uint64_t* q_full = bars;                 // [2] query tile written (once per stretch)
  uint64_t* kh_full = q_full + 2;          // [2] K tile widened
  uint64_t* vh_full = kh_full + 2;         // [2] V tile widened
  uint64_t* meta_full = vh_full + 2;       // [TMETA] page ids and scales of a tile written
  uint64_t* meta_free = meta_full + TMETA; // [TMETA] the tile's softmax is done
  uint64_t* s_full = meta_free + TMETA;    // [2 query tiles][4 steps] QK done
  uint64_t* pv_done = s_full + 8;          // [2][4] PV done
  uint64_t* p_full = pv_done + 8;          // [2][2] P stored
  uint64_t* raw_full = p_full + 4;         // [2] K codes, V codes landed
  uint64_t* raw_free = raw_full + 2;       // [2] and read
  uint64_t* seg_full = raw_free + 2;       // [2] stretch written
  uint64_t* seg_free = seg_full + 2;       // [2] every role is done with it
  uint64_t* drain = seg_free + 2;          // [2] every MMA of an issuing thread done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC + 4);
  volatile Stretch* segs = reinterpret_cast<volatile Stretch*>(sm + LY::SEG);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&kh_full[i], 4);
      mbar_init(&vh_full[i], 4);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], 4);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_free[i], 15);
      mbar_init(&drain[i], 1);
    }
    for (int i = 0; i < TMETA; ++i) {
      mbar_init(&meta_full[i], 1);
      mbar_init(&meta_free[i], 8);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 14 && lane == 0) {
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
  SH::template prefix<TTHREADS>(a, pre, reinterpret_cast<long long*>(sm + LY::SUMS), false);
  const int H = a.pv.H, G = a.pv.G;
  const long long total = pre[a.pb.n_seqs] * H;
  long long stretch = (total + gridDim.x - 1) / gridDim.x;
  if (stretch < 6) stretch = 6;
  const int worker = blockIdx.x;
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  Place pl;
  if (warp == 13 && u < end) pl = find_place<SH, TTR, KT>(a, pre, u);
  __syncthreads();                         // the prefix sums' room is the query tiles' now

  // ``done``: tiles of the line that a role has behind it; it gives the stage
  // and phase of every barrier of a tile or of its steps.  A wait tells a phase
  // only from the one before it, so no barrier may complete twice before all of
  // its waiters have seen the first: a role that has nothing to do in a tile
  // still waits, and arrives where the next phase needs that it has.
  if (warp < 8) {
    // ======================================================== softmax
    reg_inc<176>();
    const int t = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + TM_S + 128 * t;
    const uint32_t o_at = tmem + lanes + TM_O + 128 * t;
    int done = 0, steps = 0;               // steps: of P's barriers
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
      if (n > 0 && rows > 0) {
        // ------------------------------------------------------ queries
        // a warp its own 32 rows, each by L lanes of 16 channels; four turns'
        // loads in flight
        constexpr int L = D / 16;
        constexpr int RSTEP = 32 / L;                    // rows per turn
        constexpr int BATCH = 4;
        static_assert(32 % (RSTEP * BATCH) == 0);
        const int ql = tid % L;
        const int rr0 = 32 * (warp & 3) + lane / L;
        float* rfs = reinterpret_cast<float*>(sm + LY::RF) + t * TM_ROWS;
        const RopeLane rl = rope_lane(a.pv, ql * 8);
        bool bad = false;
        // the token and head of a row, carried from one turn to the next
        const int step_i = RSTEP / G, step_g = RSTEP - step_i * G;
        int qi = (r0 + rr0) / G, qg = r0 + rr0 - qi * G;
        const T* qp = static_cast<const T*>(a.q) + (size_t)head0 * D + ql * 16;
#pragma unroll 1
        for (int rr = rr0; rr < 32 * (warp & 3) + 32; rr += RSTEP * BATCH) {
          uint4 w0[BATCH], w1[BATCH];
          float2 cs[BATCH][8];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const bool on = rr + k * RSTEP < rows;       // rows past the last: zeros
            w0[k] = w1[k] = make_uint4(0, 0, 0, 0);
            if (on) {
              const uint4* src = reinterpret_cast<const uint4*>(qp + (s0 + qi) * a.q_stride + qg * D);
              w0[k] = __ldg(src);
              w1[k] = __ldg(src + 1);
            }
            rope_load(a.pv, rl, a.q_pos + (size_t)(s0 + (on ? qi : 0)) * a.pv.n_axes, cs[k], bad);
            qi += step_i;
            qg += step_g;
            if (qg >= G) {
              qg -= G;
              ++qi;
            }
          }
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
        // ------------------------------------------------------ key tiles
        // steps below j_lo and from j_hi on hold keys that some row of the warp does not see
        const int j_hi = __reduce_min_sync(0xFFFFFFFFu, hi >= k0 * KT ? (hi - k0 * KT) / STEP_KEYS : 0);
        const int j_lo = __reduce_max_sync(0xFFFFFFFFu, (lo - k0 * KT + STEP_KEYS - 1) / STEP_KEYS);
        float rf = 0.0f;
#pragma unroll 1
        for (int j = 0; j < n * SPT; ++j, ++steps) {
          const int x = done * SPT + j;
          if (!warp_wait(&s_full[4 * t + (x & 3)], (x >> 2) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sb = s_at + 64 * (x & 1);
          uint32_t xr[64];
          tmem_ld_32x32b_x64(sb, xr);
          float* s = reinterpret_cast<float*>(xr);
          if (j == 0) rf = rfs[row];       // written before q_full, which S waited for
          const int stage = (x / SPT) % TMETA;
          const float4* meta = reinterpret_cast<const float4*>(sm + LY::META) + stage * NG + (x % SPT) * 4;
          if (j >= j_hi || j < j_lo) {
            const int key0 = k0 * KT + j * STEP_KEYS;
#pragma unroll
            for (int k = 0; k < STEP_KEYS; ++k)
              if (key0 + k >= hi || key0 + k < lo) s[k] = -INFINITY;
          }
          float4 mt[4];
          float f[4], my = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mt[q] = meta[q];
            f[q] = fmaxf(rf * mt[q].x, 0x1p-100f);       // never 0, so that a masked score stays -inf
            const float* v = s + 16 * q;
            const float a0 = max3f(v[0], v[1], v[2]), a1 = max3f(v[3], v[4], v[5]), a2 = max3f(v[6], v[7], v[8]);
            const float a3 = max3f(v[9], v[10], v[11]), a4 = max3f(v[12], v[13], fmaxf(v[14], v[15]));
            my = fmaxf(my, fmaf(max3f(max3f(a0, a1, a2), a3, a4), f[q], mt[q].y));
          }
          if (__any_sync(0xFFFFFFFFu, my > m + kRaise)) {
            // rare after a row's first keys: what was summed with the old
            // maximum is brought to the new one
            const float mn = my > m + kRaise ? my : m;
            const float al = mn > m ? ex2f(m - mn) : 1.0f;     // 0 for the row's first keys
            m = mn;
            l *= al;
            if (j > 0) {
              if (!warp_wait(&pv_done[4 * t + ((x - 1) & 3)], ((x - 1) >> 2) & 1, abort_flag)) ok = false;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < D; k += 16) {
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
          for (int c = 0; c < 2; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int q = 2 * c + e;
              const float ad = mt[q].y + sub;
              float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float2 y = fma2(make_float2(s[16 * q + 2 * k], s[16 * q + 2 * k + 1]), make_float2(f[q], f[q]),
                                make_float2(ad, ad));
                y.x = ex2f(y.x);
                y.y = ex2f(y.y);
                sum = add2(sum, y);
                p[8 * e + k] = cvt_f16x2(y.x, y.y);
              }
              l = fmaf(sum.x + sum.y, mt[q].z, l);
            }
            tmem_st_32x32b_x16(sb + 16 * c, p);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_full[2 * t + (steps & 1)]);
            if (x % SPT == SPT - 1) mbar_arrive(&meta_free[stage]);
          }
          if (!ok) break;
        }
      } else {
        for (int j = 0; ok && j < n * SPT; ++j, ++steps) {
          const int x = done * SPT + j;
          ok = warp_wait(&s_full[4 * t + (x & 3)], (x >> 2) & 1, abort_flag);
          if (lane == 0) {
            mbar_arrive(&p_full[2 * t + (steps & 1)]);
            if (x % SPT == SPT - 1) mbar_arrive(&meta_free[(x / SPT) % TMETA]);
          }
        }
      }
      done += n;
      if (ok && n > 0) {
        const int x = done * SPT - 1;
        ok = warp_wait(&pv_done[4 * t + (x & 3)], (x >> 2) & 1, abort_flag);
      }
      if (!ok) break;
      tc_fence_after();
      // -------------------------------------------------------- results
      // A thread has a row, memory wants rows side by side in a warp: through
      // the warp's own rows of the query tile, which every MMA is done with.
      if (rows > 0) {
        const bool whole = flags & STRETCH_WHOLE;
        const size_t at_row = (size_t)(2 * worker + (flags & STRETCH_HEAD ? 1 : 0)) * TTR + t * TM_ROWS + row;
        uint8_t* own = sm + LY::Q + t * NQ * LY::QB + 32 * (warp & 3) * 128;
        auto put = [&](int c, uint4 v) {                 // 16-byte chunk c of the thread's row
          *reinterpret_cast<uint4*>(own + (c >> 3) * (TM_ROWS * 128) + lane * 128 + (((c & 7) ^ (lane & 7)) << 4)) = v;
        };
        auto flush = [&](auto chunks, void* dst) {       // that many chunks of every row to the row's dst
          constexpr int N = decltype(chunks)::value;
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < N; ++i) {
            const int rr = i * (32 / N) + lane / N, c = lane % N;
            const unsigned long long p = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(dst), rr);
            const uint4 v = *reinterpret_cast<const uint4*>(own + (c >> 3) * (TM_ROWS * 128) + rr * 128 +
                                                            (((c & 7) ^ (rr & 7)) << 4));
            if (p) reinterpret_cast<uint4*>(p)[c] = v;
          }
          __syncwarp();
        };
        if (whole) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (n > 0) {
              tmem_ld_32x32b_x32(o_at + c, o);
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
          T* dst = static_cast<T*>(a.out) + (s0 + i) * a.out_stride + (size_t)(head0 + (live ? r0 + row - i * G : 0)) * D;
          flush(std::integral_constant<int, D / 8>{}, live ? dst : nullptr);
        } else {
          if (live) a.tiles.ml[at_row] = make_float2(m, l);
          if (n > 0) {
            // half of the row at a time: a row has D * 2 bytes there
#pragma unroll 1
            for (int half = 0; half < D; half += D / 2) {
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_at + half + c, o);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  put(c / 4 + k, make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
              }
              flush(std::integral_constant<int, D / 8>{}, live ? a.tiles.o + at_row * D + half : nullptr);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
    }
  } else if (warp < 12) {
    // ======================================================== K, V
    reg_dec<104>();
    const int ct = tid - 256;
    constexpr int CH = D / 16;                           // 16-byte code chunks of a row
    constexpr int NT = KT * CH / 128;                    // chunks of K, and of V, per thread
    constexpr int STEP = KT / NT;                        // rows per round of the 128 threads
    const int sl0 = CH == 8 ? 8 * (ct >> 6) + (ct & 7) : 8 * (ct >> 5) + (ct & 7);
    const int ch = (ct >> 3) & (CH - 1);
    int done = 0;
    bool ok = true;
    for (int sg = 0; ok; ++sg) {
      if (!warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
      const volatile Stretch& seg = segs[sg & 1];
      if (!(seg.flags & STRETCH_SOME)) break;
      const int k0 = seg.k0, n = seg.k1 - k0, lo = seg.lo, hi = seg.hi;
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
          const uint8_t* src = sm + LY::RAW + v * KT * D;
          uint4 reg[NT];
#pragma unroll
          for (int it = 0; it < NT; ++it) reg[it] = *reinterpret_cast<const uint4*>(src + raw_chunk<D>(it * STEP + sl0, ch));
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_free[v]);
          const int key0 = (k0 + j) * KT;
          if (v && (key0 + KT > hi || key0 < lo)) {
            // values that no query sees: zeros, whatever their page holds (a
            // NaN code too); their scores are masked
#pragma unroll
            for (int it = 0; it < NT; ++it) {
              const int key = key0 + it * STEP + sl0;
              if (key >= hi || key < lo) reg[it] = make_uint4(0, 0, 0, 0);
            }
          }
          if (g >= 2) {
            // the last step of the tile before the last, of both query tiles
            const int x = (g - 1) * SPT - 1;
            uint64_t* free = (v ? pv_done : s_full) + (x & 3);
            ok = warp_wait(free, (x >> 2) & 1, abort_flag) && warp_wait(free + 4, (x >> 2) & 1, abort_flag);
            if (!ok) break;
          }
          uint8_t* dst = sm + (v ? LY::VH : LY::KH) + buf * LY::KB + (ch >> 2) * (KT * 128);
          const int cc = (2 * ch) & 7;
#pragma unroll
          for (int it = 0; it < NT; ++it) {
            const int sl = it * STEP + sl0;
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
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive((v ? vh_full : kh_full) + buf);
        }
      }
      done += n;
      if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
    }
  } else {
    reg_dec<56>();
    if (warp == 12 || warp == 15) {
      // ====================================================== MMA issue
      if (lane == 0) {
        constexpr uint32_t idesc_qk = make_idesc(0, 0, 0, 0, TM_ROWS, STEP_KEYS);
        constexpr uint32_t idesc_pv = make_idesc(0, 0, 0, 1, TM_ROWS, D);
        const int t = warp == 12 ? 0 : 1;
        const uint32_t q = smem_u32(sm + LY::Q) + t * NQ * LY::QB;
        const uint32_t kh0 = smem_u32(sm + LY::KH), vh0 = smem_u32(sm + LY::VH);
        const uint32_t o = tmem + TM_O + 128 * t, s = tmem + TM_S + 128 * t;
        uint32_t nq = 0, np = 0;                         // stretches of this query tile, and steps, so far
        int done = 0;
        // S of step x: 64 channels (a column block of 128-byte rows) per turn of the loop
        auto qk = [&](int x) {
          const uint32_t kh = kh0 + ((x / SPT) & 1) * LY::KB + (x % SPT) * (STEP_KEYS * 128);
#pragma unroll 1
          for (int c = 0; c < NQ * (D / 64); ++c) {
            const int block = c & (D / 64 - 1), part = c / (D / 64);
            mma4_f16_ss(s + 64 * (x & 1), make_sdesc_sw128(q + part * LY::QB + block * (TM_ROWS * 128), 16, 1024),
                        make_sdesc_sw128(kh + block * (KT * 128), 16, 1024), idesc_qk, c);
          }
        };
        auto k_ready = [&](int x) -> bool {              // the tile of step x, at its first step
          const int g = x / SPT;
          return x % SPT != 0 || mbar_wait(&kh_full[g & 1], (g >> 1) & 1, abort_flag);
        };
        bool ok = true;
        for (int sg = 0; ok; ++sg) {
          if (!mbar_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
          const volatile Stretch& seg = segs[sg & 1];
          if (!(seg.flags & STRETCH_SOME)) break;
          const int ns = (seg.k1 - seg.k0) * SPT;
          const bool on = seg.n * G - seg.tile * TTR > t * TM_ROWS;   // the query tile has rows
          if (ns > 0 && on && !mbar_wait(&q_full[t], nq++ & 1, abort_flag)) break;
          // QK of the first two steps; then PV of a step and QK of the one two after it
#pragma unroll 1
          for (int j = -2; j < ns; ++j) {
            const int x = done * SPT + j;
            if (j >= 0) {
              const int g = x / SPT;
              ok = (x % SPT != 0 || mbar_wait(&vh_full[g & 1], (g >> 1) & 1, abort_flag)) &&
                   mbar_wait(&p_full[2 * t + (np & 1)], (np >> 1) & 1, abort_flag);
              if (!ok) break;
              ++np;
              tc_fence_after();
              if (on)
                mma4_f16_ts(o, s + 64 * (x & 1),
                            make_sdesc_sw128(vh0 + (g & 1) * LY::KB + (x % SPT) * (STEP_KEYS * 128), KT * 128, 1024),
                            idesc_pv, j > 0);
              mma_commit(&pv_done[4 * t + (x & 3)]);
            }
            if (j + 2 < ns) {
              ok = k_ready(x + 2);
              if (!ok) break;
              tc_fence_after();
              if (on) qk(x + 2);
              mma_commit(&s_full[4 * t + ((x + 2) & 3)]);
            }
          }
          done += seg.k1 - seg.k0;
          mbar_arrive(&seg_free[sg & 1]);
        }
        // every MMA issued so far is done before the block releases its tensor memory
        mma_commit(&drain[t]);
        mbar_wait(&drain[t], 0, nullptr, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 13) {
      // ====================================================== the line of work
      PieceRec rec = {};
      int done = 0, sg = 0;
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
        auto group = [&](int k, int& pg, float& sv) {
          const int key = k * KT + lane * 16;
          pg = kNone;
          sv = 0.0f;
          if (lane < NG && k < k1 && key < pl.t.hi && key + 16 > pl.t.lo) {
            pg = __ldg(tab + (key >> a.pv.p_shift));
            if (pg < 0 || pg >= a.pv.n_pages) {
              atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
              pg = 0;
            }
            sv = __ldg(a.pv.v_scale + (size_t)pg * H + pl.h);
          }
          float mx = sv;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
          return mx;
        };
        for (int k = k0; k < k1; ++k) {
          const int g = done + k - k0;
          int pg;
          float sv;
          float mx = group(k, pg, sv);
          const float sk = pg != kNone ? __ldg(a.pv.k_scale + (size_t)pg * H + pl.h) : 0.0f;
          if (mx == 0.0f && near == 0.0f) {
            int unused;
            float v;
            for (int s = k + 1; mx == 0.0f && s < k1; ++s) mx = group(s, unused, v);
            if (mx == 0.0f) mx = 1.0f;
          }
          if (mx > 0.0f) near = mx;
          if (g >= TMETA && !warp_wait(&meta_free[g % TMETA], ((g - TMETA) / TMETA) & 1, abort_flag)) {
            ok = false;
            break;
          }
          if (lane < NG) {
            const float v = sv > 0.0f ? sv : near;
            reinterpret_cast<float4*>(sm + LY::META)[(g % TMETA) * NG + lane] =
                make_float4(sk, __log2f(v), 1.0f / v, __int_as_float(pg));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&meta_full[g % TMETA]);
        }
        done += k1 - k0;
        if (u == pl.at && end < item_end) 
          rec = {min(pl.s.n * G - pl.tile * TTR, TTR), (int)((item_end - 1) / stretch), pl.h, pl.s.s0, pl.tile * TTR};
        u = min(end, item_end);
        more = u < end && next_place<SH, TTR, KT>(a, pl);
      }
      if (lane == 0) a.tiles.rec[worker] = rec;
    } else if (warp == 14) {
      // ====================================================== TMA
      // lane i a box of the tile: 32 rows of a page (16 where a page has no more)
      const int rows = a.pv.P < 32 ? a.pv.P : 32;
      const int boxes = KT / rows;
      int done = 0, issued = 0;                          // tiles; copies (K, V, K, ...)
      bool ok = true;
      for (int sg = 0; ok; ++sg) {
        if (!warp_wait(&seg_full[sg & 1], (sg >> 1) & 1, abort_flag)) break;
        const volatile Stretch& seg = segs[sg & 1];
        if (!(seg.flags & STRETCH_SOME)) break;
        const int k0 = seg.k0, n = seg.k1 - k0, h = seg.h;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int g = done + j;
          ok = warp_wait(&meta_full[g % TMETA], (g / TMETA) & 1, abort_flag);
          if (!ok) break;
          int pg = kNone;
          if (lane < boxes) {
            const int4* meta = reinterpret_cast<const int4*>(sm + LY::META) + (g % TMETA) * NG;
            pg = rows == 16 ? meta[lane].w : max(meta[2 * lane].w, meta[2 * lane + 1].w);
          }
          const int key = (k0 + j) * KT + lane * rows;
          const int y = (int)(a.pv.row0 + (((long long)pg * H + h) << a.pv.p_shift)) + (key & (a.pv.P - 1));
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, pg != kNone)) * rows * D;
          for (int v = 0; v < 2; ++v) {
            if (g >= 1 && !warp_wait(&raw_free[v], (g - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[v], bytes);
            __syncwarp();
            if (pg != kNone)
              tma_load_2d(sm + LY::RAW + v * KT * D + lane * rows * D, v ? &tmV : &tmK, &raw_full[v], 0, y);
            issued = 2 * g + v + 1;
          }
          if (!ok) break;
        }
        done += n;
        if (lane == 0) mbar_arrive(&seg_free[sg & 1]);
      }
      // after an abort: copies still in flight land in this block's shared memory
      if (*abort_flag && issued > 0) {
        mbar_wait(&raw_full[0], ((issued - 1) >> 1) & 1, nullptr, 100000000ull);
        if (issued > 1) mbar_wait(&raw_full[1], ((issued - 2) >> 1) & 1, nullptr, 100000000ull);
      }
    }
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) atomicOr(&a.pv.state[PST_ERR], DEVERR_TIMEOUT);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
template <int D, typename T>
static cudaError_t prepare_t() {
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
