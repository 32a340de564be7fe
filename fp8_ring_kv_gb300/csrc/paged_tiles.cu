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
// while the softmax of the other runs.  Tensor memory is full: S (then P) of
// both tiles and O of both.
//
// Warp roles (512 threads, registers moved from the last two groups to the softmax):
//   warps 0-3, 4-7   softmax of query tile 0, 1: one row per thread.  They also
//                    load and rotate the rows' queries and write the output
//   warps 8-11       K and V: page ids and codes of the next tile into
//                    registers, the current ones widened into shared memory;
//                    warp 8 the pages' scales
//   warp 12          MMA issue
// MMAs run in the order they are issued: QK of the next tile may overwrite
// the P that the PV before it reads.
#include "paged_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int TM_ROWS = 128;                 // rows of one MMA
constexpr int TTR = kTilesRows;              // rows of an item: two query tiles
static_assert(TTR == 2 * TM_ROWS);
constexpr int TTHREADS = 512;
constexpr int TMETA = 4;                     // scale stages
constexpr float kRaise = 8.0f;               // a row's maximum is raised when a tile exceeds it by 2^8 ...
constexpr float kTop = 6.0f;                 // ... and starts its weights at 2^6, so they stay below 2^14 in fp16

template <int D, typename T>
struct TilesLayout {
  static constexpr int NQ = std::is_same_v<T, __half> ? 2 : 1;   // fp16 parts of a query
  static constexpr int KT = NQ == 2 ? 64 : 128;                  // keys per tile
  static constexpr int QB = TM_ROWS * D * 2;                     // one part of one query tile
  static constexpr int KB = KT * D * 2;                          // one widened K or V tile
  static constexpr int Q = 0;                                    // [2 tiles][NQ]
  static constexpr int KH = Q + 2 * NQ * QB;                     // [2]
  static constexpr int VH = KH + 2 * KB;                         // [2]
  static constexpr int META = VH + 2 * KB;                       // [TMETA][KT / 16] float4 {s_k, log2 s_v, 1 / s_v, -}
  static constexpr int BAR = META + TMETA * (KT / 16) * 16;
  static constexpr int NBAR = 2 + 2 + 2 + TMETA + 4 + 4 + 2 + 1;
  static constexpr int SUMS = BAR + NBAR * 8;
  static constexpr int MISC = SUMS + 16 * 8;
  static constexpr int ALLOC = MISC + 16 + 1024;
  static_assert(ALLOC <= 232448, "shared memory of a block");
  static_assert(KH >= (kPagedMaxSeqs + 1) * 8, "the prefix sums lie in the query tiles at first");
};

template <int D, typename T>
__global__ void __launch_bounds__(TTHREADS, 1) paged_attend_tiles_kernel(const __grid_constant__ PagedAttn a) {
  using LY = TilesLayout<D, T>;
  constexpr int KT = LY::KT, NQ = LY::NQ, NG = KT / 16;
  using SH = Share<TTR, KT, 2, kRowsMax<T>, 0x7FFFFFFF>;
  constexpr uint32_t TM_S = 0, TM_O = 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR);
  uint64_t* q_full = bars;                 // [2] query tile written (once per stretch of an item)
  uint64_t* kh_full = q_full + 2;          // [2] K tile widened
  uint64_t* vh_full = kh_full + 2;         // [2] V tile widened
  uint64_t* meta_full = vh_full + 2;       // [TMETA] scales written
  uint64_t* s_full = meta_full + TMETA;    // [2 query tiles][2] QK done; of tile 1: both, and the K tile is free
  uint64_t* o_done = s_full + 4;           // [2][2] PV done; of tile 1: both, and the V tile is free
  uint64_t* p_full = o_done + 4;           // [2] P stored
  uint64_t* drain = p_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + LY::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&kh_full[i], 4);
      mbar_init(&vh_full[i], 4);
      mbar_init(&p_full[i], 4);
    }
    for (int i = 0; i < TMETA; ++i) mbar_init(&meta_full[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
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
  const long long begin = min(total, stretch * worker), end = min(total, begin + stretch);
  Place pl;
  if (begin < end) pl = find_place<SH, TTR, KT>(a, pre, begin);
  __syncthreads();                         // the prefix sums' room is the query tiles' now
  long long u = begin;
  // one step along the line: the stretch of the current item, its key tiles [k0, k1)
  int k0 = 0, k1 = 0;
  bool whole = false, heads = false;       // heads: the item begins here
  long long item_end = 0;
  auto cut_item = [&]() {
    item_end = pl.at + pl.units;
    const int n = pl.t.t1 - pl.t.t0;
    k0 = pl.t.t0 + (int)max(0ll, min((long long)n, u - pl.at - 2));
    k1 = pl.t.t0 + (int)max(0ll, min((long long)n, min(end, item_end) - pl.at - 2));
    heads = u == pl.at;
    whole = heads && end >= item_end;
  };
  auto advance = [&]() -> bool {
    u = min(end, item_end);
    return u < end && next_place<SH, TTR, KT>(a, pl);
  };
  // tiles of the whole line that this block has done: parity and stage of every barrier
  int done = 0;
  const bool work = begin < end;

  if (warp < 8) {
    // ======================================================== softmax
    reg_inc<176>();
    const int t = warp >> 2;
    const int row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + TM_S + 128 * t;
    const uint32_t o_at = tmem + lanes + TM_O + 128 * t;
    bool ok = true;
    for (bool more = work; more && ok; more = advance()) {
      cut_item();
      const int rows = pl.s.n * G;
      const int n = k1 - k0;
      const int r = pl.tile * TTR + t * TM_ROWS + row;
      if (pl.tile * TTR + t * TM_ROWS >= rows) {
        // nothing in this query tile: keep step with the barriers, whose waits
        // tell one phase from the next only
        for (int j = 0; ok && j < n; ++j)
          ok = warp_wait(&s_full[2 * t + ((done + j) & 1)], ((done + j) >> 1) & 1, abort_flag);
        done += n;
        if (ok && n > 0) ok = warp_wait(&o_done[2 * t + ((done - 1) & 1)], ((done - 1) >> 1) & 1, abort_flag);
        continue;
      }
      const bool live = r < rows;
      const int i = live ? r / G : 0;
      const int hq = pl.h * G + (live ? r - i * G : 0);
      const int at = pl.s.len - pl.s.n + i;            // the row's own index
      const int hi = !live ? 0x7FFFFFFF : a.causal ? at + 1 : pl.s.len;
      const int lo = live && a.window > 0 ? at - a.window + 1 : 0;
      float m = -INFINITY, l = 0.0f;
      if (n > 0) {
        // ------------------------------------------------------ the row's query
        float x[D];
        float amax = 0.0f;
        if (live) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (pl.s.s0 + i) * a.q_stride +
                                                            (size_t)hq * D);
          const int32_t* pr = a.q_pos + (size_t)(pl.s.s0 + i) * a.pv.n_axes;
          bool bad = false;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) load8_f32<T>(__ldg(src + c), x + 8 * c);
#pragma unroll
          for (int k = 0; k < D / 2; ++k) {
            const float2 cs = rope_cs(a.pv, pr, k, bad);
            rope_pair(x[2 * k], x[2 * k + 1], cs.x, cs.y);
          }
          if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
        } else {
#pragma unroll
          for (int k = 0; k < D; ++k) x[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < D; ++k) amax = fmaxf(amax, fabsf(x[k]));
        const int ex = amax > 0.0f ? max(-120, min(120, ilogbf(amax))) : 0;
        const float down = ldexpf(1.0f, -ex);
        const float rf = ldexpf(a.scale_log2, ex);
        uint8_t* qs = sm + LY::Q + t * NQ * LY::QB + row * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t w[4], v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x0 = x[8 * c + 2 * k] * down, x1 = x[8 * c + 2 * k + 1] * down;
            w[k] = cvt_f16x2(x0, x1);
            if constexpr (NQ == 2) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
              v[k] = cvt_f16x2(x0 - f.x, x1 - f.y);
            }
          }
          uint8_t* dst = qs + (c >> 3) * (TM_ROWS * 128) + (((c & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          if constexpr (NQ == 2) *reinterpret_cast<uint4*>(dst + LY::QB) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
        // ------------------------------------------------------ key tiles
        for (int j = 0; j < n; ++j) {
          const int g = done + j;
          if (!warp_wait(&meta_full[g % TMETA], (g / TMETA) & 1, abort_flag) ||
              !warp_wait(&s_full[2 * t + (g & 1)], (g >> 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t xr[KT];
          if constexpr (KT == 128) tmem_ld_32x32b_x128(s_at, xr);
          else tmem_ld_32x32b_x64(s_at, xr);
          float* s = reinterpret_cast<float*>(xr);
          const float4* meta = reinterpret_cast<const float4*>(sm + LY::META) + (g % TMETA) * NG;
          const int key0 = (k0 + j) * KT;
          if (__any_sync(0xFFFFFFFFu, key0 + KT > hi || key0 < lo)) {
#pragma unroll
            for (int c = 0; c < KT; ++c)
              if (key0 + c >= hi || key0 + c < lo) s[c] = -INFINITY;
          }
          float f[NG];
          float my = -INFINITY;
#pragma unroll
          for (int q = 0; q < NG; ++q) {
            const float4 mt = meta[q];
            // never 0, so that a masked score stays -inf
            f[q] = fmaxf(rf * mt.x, 0x1p-100f);
            float* sq = s + 16 * q;
            const float a0 = max3f(sq[0], sq[1], sq[2]), a1 = max3f(sq[3], sq[4], sq[5]);
            const float a2 = max3f(sq[6], sq[7], sq[8]), a3 = max3f(sq[9], sq[10], sq[11]);
            const float a4 = max3f(sq[12], sq[13], fmaxf(sq[14], sq[15]));
            my = fmaxf(my, fmaf(fmaxf(max3f(a0, a1, a2), fmaxf(a3, a4)), f[q], mt.y));
          }
          if (__any_sync(0xFFFFFFFFu, my > m + kRaise)) {
            const float mn = my > m + kRaise ? my : m;
            const float al = mn > m ? ex2f(m - mn) : 1.0f;     // 0 for the row's first keys
            m = mn;
            l *= al;
            if (j > 0) {
              if (!warp_wait(&o_done[2 * t + ((g - 1) & 1)], ((g - 1) >> 1) & 1, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(o_at + c, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                tmem_st_32x32b_x16(o_at + c, o);
              }
            }
          }
          const float sub = m == -INFINITY ? 0.0f : kTop - m;
#pragma unroll
          for (int q = 0; q < NG; q += 2) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 mt = meta[q + e];
              const float2 ff = make_float2(f[q + e], f[q + e]), ad = make_float2(mt.y + sub, mt.y + sub);
              float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                float2 y = fma2(make_float2(s[16 * (q + e) + 2 * c], s[16 * (q + e) + 2 * c + 1]), ff, ad);
                y.x = ex2f(y.x);
                y.y = ex2f(y.y);
                sum = add2(sum, y);
                p[8 * e + c] = cvt_f16x2(y.x, y.y);
              }
              l = fmaf(sum.x + sum.y, mt.z, l);
            }
            tmem_st_32x32b_x16(s_at + 8 * q, p);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t]);
        }
        if (ok && !warp_wait(&o_done[2 * t + ((done + n - 1) & 1)], ((done + n - 1) >> 1) & 1, abort_flag)) ok = false;
        if (!ok) break;
        tc_fence_after();
      }
      done += n;
      // -------------------------------------------------------- results
      const size_t at_row = (size_t)(2 * worker + (heads ? 1 : 0)) * TTR + t * TM_ROWS + row;
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      T* dst = static_cast<T*>(a.out) + (pl.s.s0 + i) * a.out_stride + (size_t)hq * D;
      if (!whole && live) a.tiles.ml[at_row] = make_float2(m, l);
      if (whole || n > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld_32x32b_x32(o_at + c, o);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0u;
          }
          if (live && whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack2<T>(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (live) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(a.tiles.o + at_row * D + c + 4 * k) =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
      }
      tc_fence_before();
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
    const bool scales = warp == 8 && lane < NG;
    constexpr int kNone = -0x7FFFFFFF - 1;               // no query sees the key
    int id[NT], gid = kNone;
    uint4 kr[NT], vr[NT];
    float near = 0.0f;
    bool ok = true;
    for (bool more = work; more && ok; more = advance()) {
      cut_item();
      const int32_t* tab = a.pb.table + pl.b * a.pb.table_stride;
      auto page_of = [&](int key) -> int {
        if (key >= pl.t.hi || key < pl.t.lo) return kNone;
        return __ldg(tab + (key >> a.pv.p_shift));
      };
      auto ids = [&](int k) {
#pragma unroll
        for (int it = 0; it < NT; ++it) id[it] = k < k1 ? page_of(k * KT + it * STEP + sl0) : kNone;
        if (scales) {
          // a group of 16 keys that any query sees lies in one page
          const int key = k * KT + lane * 16;
          gid = k < k1 && key < pl.t.hi && key + 16 > pl.t.lo ? __ldg(tab + (key >> a.pv.p_shift)) : kNone;
        }
      };
      auto load = [&](const uint8_t* codes, int k, uint4 (&reg)[NT]) {
#pragma unroll
        for (int it = 0; it < NT; ++it) {
          const int key = k * KT + it * STEP + sl0;
          reg[it] = make_uint4(0, 0, 0, 0);
          if (k < k1 && key < pl.t.hi && key >= pl.t.lo) {
            int pg = id[it];
            if (pg < 0 || pg >= a.pv.n_pages) {
              atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
              pg = 0;
            }
            const size_t at = (((size_t)pg * H + pl.h) << a.pv.p_shift) + (key & (a.pv.P - 1));
            reg[it] = __ldg(reinterpret_cast<const uint4*>(codes + at * D) + ch);
          }
        }
      };
      auto widen = [&](uint8_t* dst, const uint4 (&reg)[NT]) {
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
          uint8_t* at = dst + (ch >> 2) * (KT * 128) + sl * 128;
          const int cc = (2 * ch) & 7;
          *reinterpret_cast<uint4*>(at + ((cc ^ (sl & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(at + (((cc + 1) ^ (sl & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      };
      float sk = 0.0f, sv = 0.0f;
      auto load_scales = [&]() {
        sk = sv = 0.0f;
        if (scales && gid != kNone) {
          const int pg = gid < 0 || gid >= a.pv.n_pages ? 0 : gid;
          sk = __ldg(a.pv.k_scale + (size_t)pg * H + pl.h);
          sv = __ldg(a.pv.v_scale + (size_t)pg * H + pl.h);
        }
      };
      auto warp_max = [&](float v) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
        return v;
      };
      if (k0 < k1) {
        near = 0.0f;
        ids(k0);
        load(a.pv.k_codes, k0, kr);
        load(a.pv.v_codes, k0, vr);
        load_scales();
        ids(k0 + 1);
      }
      for (int k = k0; k < k1; ++k) {
        const int g = done + k - k0;
        const int buf = g & 1;
        if (warp == 8) {
          // pages of zero values take a V scale near by
          float mx = warp_max(sv);
          if (mx == 0.0f && near == 0.0f) {
            for (int s = k + 1; mx == 0.0f && s < k1; ++s) {
              const int key = s * KT + lane * 16;
              float v = 0.0f;
              if (lane < NG && key < pl.t.hi && key + 16 > pl.t.lo) {
                const int pg = __ldg(tab + (key >> a.pv.p_shift));
                if (pg >= 0 && pg < a.pv.n_pages) v = __ldg(a.pv.v_scale + (size_t)pg * H + pl.h);
              }
              mx = warp_max(v);
            }
            if (mx == 0.0f) mx = 1.0f;
          }
          if (mx > 0.0f) near = mx;
          if (lane < NG) {
            const float v = sv > 0.0f ? sv : near;
            reinterpret_cast<float4*>(sm + LY::META)[(g % TMETA) * NG + lane] =
                make_float4(sk, __log2f(v), 1.0f / v, 0.0f);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&meta_full[g % TMETA]);
        }
        if (g >= 2 && !warp_wait(&s_full[2 + buf], ((g - 2) >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        widen(sm + LY::KH + buf * LY::KB, kr);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kh_full[buf]);
        load(a.pv.k_codes, k + 1, kr);
        if (g >= 2 && !warp_wait(&o_done[2 + buf], ((g - 2) >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        widen(sm + LY::VH + buf * LY::KB, vr);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vh_full[buf]);
        load(a.pv.v_codes, k + 1, vr);
        load_scales();
        ids(k + 2);
      }
      done += k1 - k0;
    }
  } else {
    // ======================================================== MMA issue
    reg_dec<56>();
    if (warp == 12 && lane == 0) {
      constexpr uint32_t idesc_qk = make_idesc(0, 0, 0, 0, TM_ROWS, KT);
      constexpr uint32_t idesc_pv = make_idesc(0, 0, 0, 1, TM_ROWS, D);
      const uint32_t q0 = smem_u32(sm + LY::Q), kh0 = smem_u32(sm + LY::KH), vh0 = smem_u32(sm + LY::VH);
      int nq[2] = {0, 0}, np[2] = {0, 0};                // stretches and tiles of each query tile so far
      auto qk = [&](int t, int g) {
#pragma unroll
        for (int part = 0; part < NQ; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ss(tmem + TM_S + 128 * t,
                       make_sdesc_sw128(q0 + (t * NQ + part) * LY::QB + (kk >> 2) * (TM_ROWS * 128) + (kk & 3) * 32, 16, 1024),
                       make_sdesc_sw128(kh0 + (g & 1) * LY::KB + (kk >> 2) * (KT * 128) + (kk & 3) * 32, 16, 1024),
                       idesc_qk, part > 0 || kk > 0 ? 1u : 0u);
      };
      bool ok = true;
      for (bool more = work; more && ok; more = advance()) {
        cut_item();
        const int n = k1 - k0;
        if (n <= 0) continue;
        const bool two = pl.s.n * G - pl.tile * TTR > TM_ROWS;
        ok = mbar_wait(&q_full[0], nq[0]++ & 1, abort_flag) && (!two || mbar_wait(&q_full[1], nq[1]++ & 1, abort_flag)) &&
             mbar_wait(&kh_full[done & 1], (done >> 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        qk(0, done);
        mma_commit(&s_full[0 + (done & 1)]);
        if (two) qk(1, done);
        mma_commit(&s_full[2 + (done & 1)]);
        for (int j = 0; j < n && ok; ++j) {
          const int g = done + j;
          for (int t = 0; t < 2; ++t) {
            const bool on = t == 0 || two;
            if (on) {
              ok = mbar_wait(&p_full[t], np[t]++ & 1, abort_flag) &&
                   (t == 1 || mbar_wait(&vh_full[g & 1], (g >> 1) & 1, abort_flag));
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                mma_f16_ts(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t + kk * 8,
                           make_sdesc_sw128(vh0 + (g & 1) * LY::KB + kk * 16 * 128, KT * 128, 1024), idesc_pv,
                           j > 0 || kk > 0 ? 1u : 0u);
            }
            mma_commit(&o_done[2 * t + (g & 1)]);
            if (j + 1 < n) {
              if (t == 0) {
                ok = mbar_wait(&kh_full[(g + 1) & 1], ((g + 1) >> 1) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
              }
              if (on) qk(t, g + 1);
              mma_commit(&s_full[2 * t + ((g + 1) & 1)]);
            }
          }
        }
        done += n;
      }
      // every MMA issued so far is done before the block releases its tensor memory
      mma_commit(drain);
      mbar_wait(drain, 0, nullptr, 100000000ull);
    }
  }
  __syncthreads();
  if (tid == 0) {
    // the item that this block began and did not end
    PieceRec rec = {-1, 0, 0, 0};
    if (work) {
      // replay of the last step: warp 0 has walked the line to its end
      if (item_end > end && heads) rec = {pl.b, pl.h, pl.tile, (int)((item_end - 1) / stretch)};
    }
    a.tiles.rec[worker] = rec;
    if (*abort_flag) atomicOr(&a.pv.state[PST_ERR], DEVERR_TIMEOUT);
  }
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
static cudaError_t tiles_t(const PagedAttn& a, int blocks, cudaStream_t st) {
  return launch_pdl(paged_attend_tiles_kernel<D, T>, dim3(blocks), dim3(TTHREADS), TilesLayout<D, T>::ALLOC, st, a);
}

cudaError_t launch_paged_tiles(const PagedAttn& a, bool f16, int blocks, cudaStream_t st) {
  if (a.pv.D == 64) return f16 ? tiles_t<64, __half>(a, blocks, st) : tiles_t<64, __nv_bfloat16>(a, blocks, st);
  return f16 ? tiles_t<128, __half>(a, blocks, st) : tiles_t<128, __nv_bfloat16>(a, blocks, st);
}

}  // namespace kvring_dev
