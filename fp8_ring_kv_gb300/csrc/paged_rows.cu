// paged_attend_rows: attention of few query rows over a paged FP8 cache.
//
//   y_t = (q . k_t) * scale * log2(e) + log2(s_v)    (k_t = code * s_k)
//   w_t = 2^(y_t - m + 8),  m the running maximum of y over the row
//   O = sum_t w_t * code(v_t),  l = sum_t w_t / s_v,  out = O / l
// The page's V scale s_v, a power of two, is an offset of the exponent: the
// weights are already those of the V codes, at most 2^8, and each sum of a
// page's weights is divided by s_v (exactly).  A page of zero V codes has
// s_v = 0; any scale serves it, and the nearest page's is taken.
//
// What bounds it: every key and value byte is read once for up to 16 rows (8 in
// fp16), and again for the next of up to 32, so HBM bandwidth, if the warps get
// through their instructions: a byte costs half a conversion and its share of
// the MMAs, whatever the number of rows.
// The codes go from memory to shared memory by TMA (32 keys and values per
// stage, a ring of stages per warp) and from there, widened to fp16 (exact),
// straight into the registers of mma.m16n8k16; a warp works by itself, with no
// barrier between warps.  tcgen05 would want 128 rows.  Measured: a batch of 64
// ragged contexts of 200 to 8,000 tokens (4 rows, 542 MB) 104 us with joining,
// 5.2 TB/s; the stretch after the first codes runs at 6.3 TB/s (93% of a copy),
// some 15 us go into the start (lengths, prefix sums, pages: 5 us) and the end.
//
// The products are S^T = K Q^T and O^T = V^T P^T: keys and channels are the
// MMA's 16 rows and the queries its 8 columns, so up to 8 query rows waste
// nothing (with the queries as rows, half of the products and of the
// accumulators were padding, two warps per sub-partition fitted, and a decoding
// batch of 64 contexts took 129 us against 103).
//
// Register layouts (lane 4 g + t): of a K tile a thread holds 16-byte chunks of
// key rows g and g + 8 (its channels are the MMA's k in a permuted order, the
// same for Q), of a V tile 16 bytes of each of four keys: byte pairs of two
// keys at one channel become the MMA's k pairs.  S^T has key g and queries
// 2 t, 2 t + 1 in a thread; movmatrix turns the weights into P^T's layout.  The
// key rows of an 8-key group are taken in the order 0 5 2 7 4 1 6 3, with
// which both patterns read 128-byte-swizzled rows without bank conflicts.
#include "paged_exact.cuh"
#include "paged_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int RK = kRowsKeys;

// NT: MMA column tiles.  1: up to 8 query rows; 2: up to 16.  fp16 queries take
// two columns a row, a high and a low part whose products are summed (an fp16
// result shows more than the 11 bits of one operand): up to 4 rows in one tile,
// the low parts in columns 4 .. 7, up to 8 in two, the low parts in the second.
template <int D, int NT>
struct RowsLayout {
  static constexpr int RW = NT == 1 ? kRowsWarps : 8;    // warps, as their registers allow
  static constexpr int NST = (NT == 1 ? 2 : 3) * (128 / D);   // stages per warp
  static constexpr int STAGE = 2 * RK * D;               // K codes, then V codes
  static constexpr int META = RW * NST * STAGE;          // per warp and stage: {s_k, log2 s_v, 1 / s_v, -} of two pages
  static constexpr int BAR = META + RW * NST * 32;
  static constexpr int PRE = BAR + RW * NST * 8;
  static constexpr int SUMS = PRE + (kPagedMaxSeqs + 1) * 8;
  static constexpr int MISC = SUMS + RW * 8;
  static constexpr int ALLOC = MISC + 16;                // the block's shared memory starts 1024-byte aligned
  static_assert(ALLOC <= 232448, "shared memory of a block");
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held as MMA fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// key row of MMA index n of an 8-key group
__device__ __forceinline__ int key_row(int n) { return ((((n >> 2) ^ n) & 1) << 2) | (n & 3); }

template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
  if constexpr (D == 128)
    return r * 128 + ((c ^ (r & 7)) << 4);
  else
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint32_t widen_lo(uint32_t w) { return cvt_e4m3x2_to_f16x2((uint16_t)(w & 0xFFFFu)); }
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) { return cvt_e4m3x2_to_f16x2((uint16_t)(w >> 16)); }

template <int D, int NT, typename T>
__global__ void __launch_bounds__(32 * RowsLayout<D, NT>::RW, 1)
    paged_attend_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const __grid_constant__ PagedAttn a) {
  using LY = RowsLayout<D, NT>;
  constexpr int NST = LY::NST, RW = LY::RW;
  constexpr bool SPLIT = std::is_same_v<T, __half>;
  constexpr bool SIDE = SPLIT && NT == 1;                // low parts beside the high ones
  constexpr int E = SPLIT ? 1 : NT;                      // tiles of query rows
  constexpr int COLS = SIDE ? 4 : 8;                     // rows of a tile
  constexpr int RT = kRowsTile<T>;                       // rows of an item, at most
  using RowsShare = Share<RT, RK, 0, 0, kRowsMax>;
  constexpr int KS = D / 16;                             // k steps of QK
  constexpr int NJ = D / 16;                             // channel tiles of O
  constexpr int DG = D / 8;                              // channels per thread
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR) + warp * NST;
  uint8_t* stages = sm + warp * NST * LY::STAGE;
  float4* metas = reinterpret_cast<float4*>(sm + LY::META) + warp * NST * 2;
  long long* pre = reinterpret_cast<long long*>(sm + LY::PRE);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + LY::MISC);
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (tid == 0) *abort_flag = 0;
  pdl_wait();
  pdl_trigger();
  RowsShare::template prefix<32 * RW>(a, pre, reinterpret_cast<long long*>(sm + LY::SUMS), blockIdx.x == 0);
  const int H = a.pv.H, G = a.pv.G;
  const int worker = blockIdx.x * RW + warp;
  const int workers = gridDim.x * RW;
  const long long total = pre[a.pb.n_seqs] * H;
  const long long stretch = quotient(total + workers - 1, workers);
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  PieceRec rec = {};
  int used = 0;                                          // stages issued so far: stage and phase of the next
  if (u < end) {
    Place pl = find_place<RowsShare, RT, RK>(a, pre, u);
    while (true) {
      const long long item_end = pl.at + pl.units;
      const int k0 = pl.t.t0 + (int)(u - pl.at);
      const int k1 = min(pl.t.t1, pl.t.t0 + (int)(min(end, item_end) - pl.at));
      const bool whole = u == pl.at && end >= item_end;
      const int row0 = pl.tile * RT, rows = min(RT, pl.s.n * G - row0);
      // ---------------------------------------------------------- pages
      // lane i holds the page ids and scales of tile base + i (two pages when
      // P = 16); v_near: a non-zero V scale near by, for pages of zeros
      int base = k0;
      int id[2] = {-1, -1};
      float sk[2] = {0.0f, 0.0f}, sv[2] = {0.0f, 0.0f};
      float v_near = 0.0f;
      ScaleSpan span;
      auto load_ids = [&](int tb, int (&ids)[2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ids[p] = -1;
          const int key = (tb + lane) * RK + p * 16;
          if (tb + lane < k1 && (p == 0 || a.pv.P == 16) && key < pl.t.hi &&
              key + (a.pv.P == 16 ? 16 : RK) > pl.t.lo) {
            ids[p] = a.pb.table[pl.b * a.pb.table_stride + (key >> a.pv.p_shift)];
            if (ids[p] < 0 || ids[p] >= a.pv.n_pages) {
              atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
              ids[p] = 0;
            }
          }
        }
      };
      auto load_scales = [&](const int (&ids)[2], float (&ks)[2], float (&vs)[2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ks[p] = ids[p] >= 0 ? a.pv.k_scale[(size_t)ids[p] * H + pl.h] : 0.0f;
          vs[p] = ids[p] >= 0 ? a.pv.v_scale[(size_t)ids[p] * H + pl.h] : 0.0f;
        }
      };
      auto near_scale = [&]() {
        auto top = [](float v) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
          return v;
        };
        span.add(sv[0]);
        span.add(sv[1]);
        float mx = top(fmaxf(sv[0], sv[1]));
        if (mx == 0.0f && v_near == 0.0f) {
          for (int tb = base + 32; mx == 0.0f && tb < k1; tb += 32) {
            int di[2];
            float dk[2], dv[2];
            load_ids(tb, di);
            load_scales(di, dk, dv);
            mx = top(fmaxf(dv[0], dv[1]));
          }
          if (mx == 0.0f) mx = 1.0f;
        }
        if (mx > 0.0f) v_near = mx;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (sv[p] == 0.0f) sv[p] = v_near;
      };
      // the codes of tiles [k, to) on their way to the next stages, each by the lane that holds its pages
      auto issue = [&](int k, int to) {
        const int mine = base + lane;
        if (mine >= k && mine < to) {
          const int st = (used + mine - k) % NST;
          uint8_t* dst = stages + st * LY::STAGE;
          if (a.pv.P == 16) {
            mbar_arrive_expect_tx(&bars[st], (uint32_t)((id[0] >= 0) + (id[1] >= 0)) * 2 * 16 * D);
#pragma unroll
            for (int p = 0; p < 2; ++p)
              if (id[p] >= 0) {
                const int y = (int)(a.pv.row0 + ((long long)id[p] * H + pl.h) * 16);
                tma_load_2d(dst + p * 16 * D, &tmK, &bars[st], 0, y);
                tma_load_2d(dst + RK * D + p * 16 * D, &tmV, &bars[st], 0, y);
              }
          } else {
            const int y = (int)(a.pv.row0 + (((long long)id[0] * H + pl.h) << a.pv.p_shift)) + ((mine * RK) & (a.pv.P - 1));
            mbar_arrive_expect_tx(&bars[st], LY::STAGE);
            tma_load_2d(dst, &tmK, &bars[st], 0, y);
            tma_load_2d(dst + RK * D, &tmV, &bars[st], 0, y);
          }
        }
        used += to - k;
      };
      auto write_meta = [&](int k, int n) {
        if (lane == k - base) {
          float4* m = metas + (n % NST) * 2;
          const int p1 = a.pv.P == 16 ? 1 : 0;
          m[0] = make_float4(sk[0], __log2f(sv[0]), 1.0f / sv[0], 0.0f);
          m[1] = make_float4(sk[p1], __log2f(sv[p1]), 1.0f / sv[p1], 0.0f);
        }
      };
      const int first = used;
      int issued = k0;
      load_ids(base, id);
      // the queries' loads ahead of the first codes, which keep the memory busy for some microseconds
      uint4 qw[E][D / 32];
      float2 cs[E][D / 8];
      bool bad = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = e * COLS + g % COLS;
        const bool live = r < rows;
        const int i = live ? (row0 + r) / G : 0;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          qw[e][2 * c] = qw[e][2 * c + 1] = make_uint4(0, 0, 0, 0);
          if (live) {
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) + (pl.s.s0 + i) * a.q_stride + (size_t)(pl.h * G + row0 + r - i * G) * D + c * 64 + t4 * 16);
            qw[e][2 * c] = src[0];
            qw[e][2 * c + 1] = src[1];
          }
          float2 part8[8];
          rope_load(a.pv, rope_lane(a.pv, c * 32 + t4 * 8), a.q_pos + (size_t)(pl.s.s0 + i) * a.pv.n_axes, part8, bad);
#pragma unroll
          for (int k = 0; k < 8; ++k) cs[e][8 * c + k] = part8[k];
        }
      }
      issued = min(k1, k0 + NST);
      issue(k0, issued);
      load_scales(id, sk, sv);
      // ---------------------------------------------------------- queries
      // row g of each tile, rotated, scaled by a power of two and rounded to
      // fp16 (an MMA operand): a bf16 query loses nothing that its output
      // could show, an fp16 one keeps a second part
      uint32_t qb[NT][KS][2];
      float rf[E][2];                                    // logit factors of rows 2 t, 2 t + 1
      int hi[E][2], lo[E][2];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t mb = 0;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) mb = __vmaxu2(mb, max8_bits(qw[e][c]));
        mb = __vmaxu2(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, 1));
        mb = __vmaxu2(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, 2));
        const int ex = query_exponent<T>(mb);
        const float down = pow2f(-ex);
        const float rfg = a.scale_log2 * pow2f(ex);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float x[8];
          load8_f32<T>(qw[e][k / 2], x);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int at = 4 * (k & 1) + 2 * f;          // of the 8 values of the chunk
            const float2 y = mul2(rope_query(x[at], x[at + 1], cs[e][2 * k + f]), make_float2(down, down));
            const uint32_t p = cvt_f16x2(y.x, y.y);
            qb[e][k][f] = p;
            if constexpr (SPLIT) {
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&p));
              const uint32_t low = cvt_f16x2(y.x - z.x, y.y - z.y);
              if constexpr (SIDE) qb[0][k][f] = g < COLS ? p : low;
              else qb[1][k][f] = low;
            }
          }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int rr = e * COLS + (2 * t4 + f) % COLS;
          const int at = pl.s.len - pl.s.n + (rr < rows ? (row0 + rr) / G : 0);   // the row's own index
          rf[e][f] = __shfl_sync(0xFFFFFFFFu, rfg, 4 * (2 * t4 + f));
          hi[e][f] = rr >= rows ? 0x7FFFFFFF : a.causal ? at + 1 : pl.s.len;
          lo[e][f] = rr < rows && a.window > 0 ? at - a.window + 1 : 0;
        }
      }
      if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
      if (k0 < k1) {
        near_scale();
        for (int k = k0; k < issued; ++k) write_meta(k, first + k - k0);
        __syncwarp();
      }
      // tiles below c_lo and from c_hi on hold keys that some row does not see
      int c_hi = pl.t.hi / RK, c_lo = (pl.t.lo + RK - 1) / RK;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          c_hi = min(c_hi, hi[e][f] / RK);
          c_lo = max(c_lo, (lo[e][f] + RK - 1) / RK);
        }
      c_hi = __reduce_min_sync(0xFFFFFFFFu, c_hi);
      c_lo = __reduce_max_sync(0xFFFFFFFFu, c_lo);
      float o[NJ][NT][4];
#pragma unroll
      for (int i = 0; i < NJ; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
      float m[E][2], l[E][2];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[e][0] = m[e][1] = -INFINITY;
        l[e][0] = l[e][1] = 0.0f;
      }
      // ---------------------------------------------------------- keys
      bool alive = true;
#pragma unroll 1
      for (int k = k0; k < k1; ++k) {
        const int n = first + (k - k0);
        const int st = n % NST;
        if (!warp_wait(&bars[st], (n / NST) & 1, abort_flag)) {
          alive = false;
          break;
        }
        const uint8_t* kc = stages + st * LY::STAGE;
        uint8_t* vc = stages + st * LY::STAGE + RK * D;
        const float4 m0 = metas[2 * st], m1 = metas[2 * st + 1];
        float c[2][NT][4];                               // 16 keys each
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) c[j][nt][0] = c[j][nt][1] = c[j][nt][2] = c[j][nt][3] = 0.0f;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            const uint4 w = *reinterpret_cast<const uint4*>(kc + code_chunk<D>(j * 16 + key_row(g), q * 4 + t4));
            const uint4 v = *reinterpret_cast<const uint4*>(kc + code_chunk<D>(j * 16 + 8 + key_row(g), q * 4 + t4));
            const uint32_t wa[4] = {w.x, w.y, w.z, w.w}, va[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = widen_lo(wa[i]), a1 = widen_lo(va[i]), a2 = widen_hi(wa[i]), a3 = widen_hi(va[i]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816(c[j][nt], a0, a1, a2, a3, qb[nt][q * 4 + i][0], qb[nt][q * 4 + i][1]);
            }
          }
        }
        // y: keys key_row(g) (+ 8) of group j, rows 2 t4 + f of tile e
        const int key0 = k * RK;
        const bool cut = k >= c_hi || k < c_lo;
        float mx[E][2];
        bool raise = false;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            mx[e][f] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int h8 = 0; h8 < 2; ++h8) {
                const int i = 2 * h8 + f;
                float s = c[j][e][i];
                if constexpr (SIDE) s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
                else if constexpr (SPLIT) s += c[j][NT - 1][i];
                float y = fmaf(s, rf[e][f] * (j ? m1.x : m0.x), j ? m1.y : m0.y);
                if (cut) {
                  const int key = key0 + j * 16 + h8 * 8 + key_row(g);
                  if (key >= hi[e][f] || key < lo[e][f] || key >= pl.t.hi) y = -INFINITY;
                }
                c[j][e][i] = y;
                mx[e][f] = fmaxf(mx[e][f], y);
              }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx[e][f] = fmaxf(mx[e][f], __shfl_xor_sync(0xFFFFFFFFu, mx[e][f], off));
            raise = raise || mx[e][f] > m[e][f];
          }
        if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const float mn = fmaxf(m[e][f], mx[e][f]);
              const float al = mn > m[e][f] ? ex2f(m[e][f] - mn) : 1.0f;     // 0 for the first keys of a row
              m[e][f] = mn;
              l[e][f] *= al;
#pragma unroll
              for (int i = 0; i < NJ; ++i) {
                o[i][e][f] *= al;
                o[i][e][2 + f] *= al;
                if constexpr (SPLIT && !SIDE) {
                  o[i][NT - 1][f] *= al;
                  o[i][NT - 1][2 + f] *= al;
                }
              }
            }
        }
        // weights, and P^T as the MMA's second operand
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float sub0 = m[e][0] == -INFINITY ? 0.0f : 8.0f - m[e][0], sub1 = m[e][1] == -INFINITY ? 0.0f : 8.0f - m[e][1];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float iv = j ? m1.z : m0.z;
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int h8 = 0; h8 < 2; ++h8) {
              const float w0 = ex2f(c[j][e][2 * h8] + sub0), w1 = ex2f(c[j][e][2 * h8 + 1] + sub1);
              s0 += w0;
              s1 += w1;
              uint32_t w = cvt_f16x2(w0, w1);
              if constexpr (SPLIT) {
                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w));
                const uint32_t low = cvt_f16x2(w0 - y.x, w1 - y.y);
                if constexpr (SIDE) w = t4 < 2 ? w : low;
                else pb[j][NT - 1][h8] = transpose8(low);
              }
              pb[j][e][h8] = transpose8(w);
            }
            l[e][0] = fmaf(s0, iv, l[e][0]);
            l[e][1] = fmaf(s1, iv, l[e][1]);
          }
        }
        // O^T += V^T P^T: k pairs are keys (row(2 t4), row(2 t4 + 1)) of either 8-key group
        if (cut) {
          // A lane looks at one key's values.  Those that no query sees become
          // zeros, whatever their page holds.  A NaN that some rows see and
          // others do not must not meet the latter's zero weights: it is left
          // out, and the sums of the rows that see it get it.
          const int key = key0 + lane;
          const bool hidden = key >= pl.t.hi || key < pl.t.lo;
          bool nan = false;
#pragma unroll 1
          for (int i = 0; i < D / 16; ++i) {
            uint4* at = reinterpret_cast<uint4*>(vc + code_chunk<D>(lane, i));
            uint4 w = *at;
            const bool n = drop_nan_codes(w.x) | drop_nan_codes(w.y) | drop_nan_codes(w.z) | drop_nan_codes(w.w);
            nan = nan || n;
            if (hidden) w = make_uint4(0, 0, 0, 0);
            if (hidden || n) *at = w;
          }
          fence_proxy_async_smem();                      // before the stage's next TMA
          const unsigned nans = __ballot_sync(0xFFFFFFFFu, nan && !hidden);
          if (nans) {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int kr = i * 8 + key_row(g);
                  if ((nans >> kr & 1) && key0 + kr < hi[e][f] && key0 + kr >= lo[e][f]) l[e][f] = __int_as_float(0x7FFFFFFF);
                }
          }
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t w[4][D / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int kr = j * 16 + (r >> 1) * 8 + key_row(2 * t4 + (r & 1));
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(vc + code_chunk<D>(kr, g));
              w[r][0] = v.x;
              w[r][1] = v.y;
              w[r][2] = v.z;
              w[r][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(vc + code_chunk<D>(kr, g >> 1) + (g & 1) * 8);
              w[r][0] = v.x;
              w[r][1] = v.y;
            }
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const uint32_t sel = f ? 0x7362 : 0x5140;
              const uint32_t x = __byte_perm(w[0][i], w[1][i], sel), y = __byte_perm(w[2][i], w[3][i], sel);
              const uint32_t a0 = widen_lo(x), a1 = widen_hi(x), a2 = widen_lo(y), a3 = widen_hi(y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_16816(o[2 * i + f][nt], a0, a1, a2, a3, pb[j][nt][0], pb[j][nt][1]);
            }
        }
        __syncwarp();                                    // every lane is done with the stage
        if (issued < k1) {
          if (issued >= base + 32) {
            base += 32;
            load_ids(base, id);
            load_scales(id, sk, sv);
            near_scale();
          }
          issue(issued, issued + 1);
          write_meta(issued, used - 1);
          ++issued;
          __syncwarp();
        }
      }
      if (!alive) {
        // copies still in flight land in this block's shared memory: wait (bounded)
        for (int n = first; n < used; ++n)
          if (n >= used - NST) mbar_wait(&bars[n % NST], (n / NST) & 1, nullptr, 100000000ull);
        break;
      }
      // ---------------------------------------------------------- results
      // a thread: rows 2 t4 + f of each tile, channels DG g ..
      const int slot = 2 * worker + (u == pl.at ? 1 : 0);
      if (span.far_apart()) {
        for (int r = 0; r < rows; ++r) {
          const int rr = row0 + r, i = rr / G;
          const size_t at_row = (size_t)slot * RT + r;
          T* dst = static_cast<T*>(a.out) + (pl.s.s0 + i) * a.out_stride + (size_t)(pl.h * G + rr - i * G) * D;
          exact_row<D, T>(a, pl.b, pl.s.s0, pl.s.n, pl.s.len, pl.h, rr, k0 * RK, k1 * RK, whole ? dst : nullptr,
                          a.rows.o + at_row * D, a.rows.ml + at_row, 8.0f);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[e][f] += __shfl_xor_sync(0xFFFFFFFFu, l[e][f], off);
            const int r = e * COLS + 2 * t4 + f;
            float v[DG];
#pragma unroll
            for (int i = 0; i < NJ; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float x = o[i][e][2 * k + f];
                if constexpr (SIDE) x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
                else if constexpr (SPLIT) x += o[i][NT - 1][2 * k + f];
                v[2 * i + k] = x;
              }
            if (r >= rows || 2 * t4 + f >= COLS) continue;
            if (whole) {
              const int i = (row0 + r) / G;
              const float inv = l[e][f] != 0.0f ? 1.0f / l[e][f] : 0.0f;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (pl.s.s0 + i) * a.out_stride +
                                                    (size_t)(pl.h * G + row0 + r - i * G) * D + g * DG);
#pragma unroll
              for (int c = 0; c < DG / 8; ++c)
                dst[c] = make_uint4(pack2<T>(v[8 * c] * inv, v[8 * c + 1] * inv), pack2<T>(v[8 * c + 2] * inv, v[8 * c + 3] * inv),
                                    pack2<T>(v[8 * c + 4] * inv, v[8 * c + 5] * inv),
                                    pack2<T>(v[8 * c + 6] * inv, v[8 * c + 7] * inv));
            } else {
              const size_t at_row = (size_t)slot * RT + r;
              float4* dst = reinterpret_cast<float4*>(a.rows.o + at_row * D + g * DG);
#pragma unroll
              for (int c = 0; c < DG / 4; ++c) dst[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
              if (g == 0) a.rows.ml[at_row] = make_float2(m[e][f], l[e][f]);
            }
          }
      }
      if (u == pl.at && end < item_end) rec = {rows, (int)quotient(item_end - 1, stretch), pl.h, pl.s.s0, row0};
      u = min(end, item_end);
      if (u >= end || !next_place<RowsShare, RT, RK>(a, pl)) break;
    }
  }
  if (lane == 0) {
    a.rows.rec[worker] = rec;
    if (*abort_flag) atomicOr(&a.pv.state[PST_ERR], DEVERR_TIMEOUT);
  }
}

// ---------------------------------------------------------------- host
template <int D, int NT, typename T>
static cudaError_t prepare_t() {
  return cudaFuncSetAttribute(paged_attend_rows_kernel<D, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsLayout<D, NT>::ALLOC);
}

template <int D>
static cudaError_t prepare_d() {
  cudaError_t e = prepare_t<D, 1, __half>();
  if (e == cudaSuccess) e = prepare_t<D, 2, __half>();
  if (e == cudaSuccess) e = prepare_t<D, 1, __nv_bfloat16>();
  return e == cudaSuccess ? prepare_t<D, 2, __nv_bfloat16>() : e;
}

cudaError_t prepare_paged_rows(int D) { return D == 128 ? prepare_d<128>() : prepare_d<64>(); }

// One column tile where no sequence of the call has more rows than it holds,
// as far as the host knows: half of the MMAs, and half as many warps again
// (64 ragged contexts, 4 rows: 108 us against 129 with two; fp16, 1 row: 42
// against 46).
static int column_tiles(const PagedAttn& a, bool f16) { return (long long)a.max_new * a.pv.G > (f16 ? 4 : 8) ? 2 : 1; }

int paged_rows_warps(const PagedAttn& a, bool f16) { return column_tiles(a, f16) == 1 ? kRowsWarps : 8; }

template <int D, int NT, typename T>
static cudaError_t rows_t(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, int blocks,
                          cudaStream_t st) {
  using LY = RowsLayout<D, NT>;
  return launch_pdl(paged_attend_rows_kernel<D, NT, T>, dim3(blocks), dim3(32 * LY::RW), LY::ALLOC, st, tmK, tmV, a);
}

template <int D>
static cudaError_t rows_d(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                          cudaStream_t st) {
  if (f16)
    return column_tiles(a, f16) == 1 ? rows_t<D, 1, __half>(a, tmK, tmV, blocks, st)
                                     : rows_t<D, 2, __half>(a, tmK, tmV, blocks, st);
  return column_tiles(a, f16) == 1 ? rows_t<D, 1, __nv_bfloat16>(a, tmK, tmV, blocks, st)
                                   : rows_t<D, 2, __nv_bfloat16>(a, tmK, tmV, blocks, st);
}

cudaError_t launch_paged_rows(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                              cudaStream_t st) {
  return a.pv.D == 64 ? rows_d<64>(a, tmK, tmV, f16, blocks, st) : rows_d<128>(a, tmK, tmV, f16, blocks, st);
}

}  // namespace kvring_dev
