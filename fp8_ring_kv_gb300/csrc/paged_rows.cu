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
// What bounds it: every key and value byte is read once for at most 16 rows,
// so HBM bandwidth.  The codes go from memory to shared memory by TMA (32 keys
// and values per stage, a ring of stages per warp) and from there, widened to
// fp16 (exact), straight into the registers of mma.m16n8k16: a warp works by
// itself, with no barrier between warps, and at 16 rows the products cost a
// fraction of what the bytes do.  tcgen05 would want 128 rows.
//
// Register layouts: a thread of lane 4g + t holds, of a K tile, 16-byte chunks
// of key row g (its channels are the MMA's k in a permuted order, the same for
// Q), and of a V tile 16 bytes of each of the four keys whose weights it
// holds: byte pairs of two keys at one channel become the MMA's k pair.  The
// key rows of an 8-key group are taken in the order 0 5 2 7 4 1 6 3, with
// which both patterns read 128-byte-swizzled rows without bank conflicts.
#include "paged_sched.cuh"
#include "launch.h"

namespace kvring_dev {

constexpr int RW = kRowsWarps, RK = kRowsKeys;
constexpr int RTHREADS = 32 * RW;

template <int D>
struct RowsLayout {
  static constexpr int NST = D == 128 ? 3 : 6;           // stages per warp
  static constexpr int STAGE = 2 * RK * D;               // K codes, then V codes
  static constexpr int META = RW * NST * STAGE;          // per warp and stage: s_k of two pages, s_v of two pages
  static constexpr int BAR = META + RW * NST * 16;
  static constexpr int PRE = BAR + RW * NST * 8;
  static constexpr int SUMS = PRE + (kPagedMaxSeqs + 1) * 8;
  static constexpr int MISC = SUMS + RW * 8;
  static constexpr int ALLOC = MISC + 16 + 1024;         // slack for 1024-byte alignment
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// key row of MMA column n of an 8-key group
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

template <int D, typename T>
__global__ void __launch_bounds__(RTHREADS, 1)
    paged_attend_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const __grid_constant__ PagedAttn a) {
  using LY = RowsLayout<D>;
  constexpr int NST = LY::NST;
  constexpr int KS = D / 16;                             // k steps of QK; also 2 x the V channel tiles per byte group
  constexpr int DG = D / 8;                              // channels of O per thread and column parity
  // MMA rows 8 .. 15: eight more query rows, or, for fp16 queries, the low
  // parts of rows 0 .. 7 (and of their weights): both parts of a product are
  // summed at the end, at no further MMA
  constexpr bool SPLIT = std::is_same_v<T, __half>;
  constexpr int RT = kRowsMax<T>, E = SPLIT ? 1 : 2;
  using RowsShare = Share<RT, RK, 0, 0, RT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + LY::BAR) + warp * NST;
  uint8_t* stages = sm + warp * NST * LY::STAGE;
  float4* metas = reinterpret_cast<float4*>(sm + LY::META) + warp * NST;
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
  RowsShare::template prefix<RTHREADS>(a, pre, reinterpret_cast<long long*>(sm + LY::SUMS), blockIdx.x == 0);
  const int H = a.pv.H, G = a.pv.G;
  const int worker = blockIdx.x * RW + warp;
  const int workers = gridDim.x * RW;
  const long long total = pre[a.pb.n_seqs] * H;
  const long long stretch = (total + workers - 1) / workers;
  long long u = min(total, stretch * worker);
  const long long end = min(total, u + stretch);
  PieceRec rec = {-1, 0, 0, 0};
  int used = 0;                                          // stages issued so far: stage and phase of the next
  if (u < end) {
    Place pl = find_place<RowsShare, RT, RK>(a, pre, u);
    while (true) {
      const long long item_end = pl.at + pl.units;
      const int k0 = pl.t.t0 + (int)(u - pl.at);
      const int k1 = min(pl.t.t1, pl.t.t0 + (int)(min(end, item_end) - pl.at));
      const bool whole = u == pl.at && end >= item_end;
      const int rows = pl.s.n * G;
      // ---------------------------------------------------------- queries
      // rows g and g + 8 of the tile, rotated, scaled by a power of two to
      // below 2 and rounded to fp16 (an MMA operand): a bf16 query loses
      // nothing that its output could show, an fp16 one keeps a second part
      uint32_t qa[KS][4];
      float rf[E];
      int hi[E], lo[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = pl.tile * RT + g + 8 * e;
        const bool live = r < rows;
        const int i = live ? r / G : 0;
        uint4 w[D / 32];
        float2 cs[D / 8];
        uint32_t mb = 0;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          w[2 * c] = w[2 * c + 1] = make_uint4(0, 0, 0, 0);
          if (live) {
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(a.q) + (pl.s.s0 + i) * a.q_stride + (size_t)(pl.h * G + r - i * G) * D + c * 64 + t4 * 16);
            w[2 * c] = __ldg(src);
            w[2 * c + 1] = __ldg(src + 1);
          }
          float2 part[8];
          rope_load(a.pv, rope_lane(a.pv, c * 32 + t4 * 8), a.q_pos + (size_t)(pl.s.s0 + i) * a.pv.n_axes, part, bad);
#pragma unroll
          for (int k = 0; k < 8; ++k) cs[8 * c + k] = part[k];
          mb = __vmaxu2(mb, __vmaxu2(max8_bits(w[2 * c]), max8_bits(w[2 * c + 1])));
        }
        if (bad) atomicOr(&a.pv.state[PST_ERR], DEVERR_POS_RANGE);
        mb = __vmaxu2(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, 1));
        mb = __vmaxu2(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, 2));
        const int ex = query_exponent<T>(mb);
        const float down = pow2f(-ex);
        rf[e] = a.scale_log2 * pow2f(ex);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float x[8];
          load8_f32<T>(w[k / 2], x);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int at = 4 * (k & 1) + 2 * f;          // of the 8 values of the chunk
            const float2 y = mul2(rope_query(x[at], x[at + 1], cs[2 * k + f]), make_float2(down, down));
            const uint32_t p = cvt_f16x2(y.x, y.y);
            qa[k][2 * f + e] = p;
            if constexpr (SPLIT) {
              const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&p));
              qa[k][2 * f + 1] = cvt_f16x2(y.x - z.x, y.y - z.y);
            }
          }
        }
        const int at = pl.s.len - pl.s.n + i;            // the row's own index
        hi[e] = !live ? 0x7FFFFFFF : a.causal ? at + 1 : pl.s.len;
        lo[e] = live && a.window > 0 ? at - a.window + 1 : 0;
      }
      float o[DG][4];
#pragma unroll
      for (int i = 0; i < DG; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
      float m[E], l[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.0f;
      }

      // ---------------------------------------------------------- pages
      // lane i holds the page ids and scales of tile base + i (two pages when
      // P = 16); v_near: a non-zero V scale near by, for pages of zeros
      int base = k0 - 32;
      int id[2] = {-1, -1};
      float sk[2] = {0, 0}, sv[2] = {0, 0};
      float v_near = 0.0f;
      auto load_pages = [&](int tb, int (&ids)[2], float (&ks)[2], float (&vs)[2]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ids[p] = -1;
          ks[p] = vs[p] = 0.0f;
          const int key = (tb + lane) * RK + p * 16;
          if (tb + lane < k1 && (p == 0 || a.pv.P == 16) && key < pl.t.hi &&
              key + (a.pv.P == 16 ? 16 : RK) > pl.t.lo) {
            int pg = __ldg(a.pb.table + pl.b * a.pb.table_stride + (key >> a.pv.p_shift));
            if (pg < 0 || pg >= a.pv.n_pages) {
              atomicOr(&a.pv.state[PST_ERR], DEVERR_PAGE);
              pg = 0;
            }
            ids[p] = pg;
            ks[p] = __ldg(a.pv.k_scale + (size_t)pg * H + pl.h);
            vs[p] = __ldg(a.pv.v_scale + (size_t)pg * H + pl.h);
          }
        }
        float mx = fmaxf(vs[0], vs[1]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        return mx;
      };
      auto issue = [&](int k) {
        if (k >= base + 32) {
          base += 32;
          float mx = load_pages(base, id, sk, sv);
          if (mx == 0.0f && v_near == 0.0f) {
            for (int tb = base + 32; mx == 0.0f && tb < k1; tb += 32) {
              int di[2];
              float dk[2], dv[2];
              mx = load_pages(tb, di, dk, dv);
            }
            if (mx == 0.0f) mx = 1.0f;
          }
          if (mx > 0.0f) v_near = mx;
#pragma unroll
          for (int p = 0; p < 2; ++p)
            if (sv[p] == 0.0f) sv[p] = v_near;
        }
        const int src = k - base;
        const int p0 = __shfl_sync(0xFFFFFFFFu, id[0], src), p1 = __shfl_sync(0xFFFFFFFFu, id[1], src);
        const float4 mt = make_float4(__shfl_sync(0xFFFFFFFFu, sk[0], src), __shfl_sync(0xFFFFFFFFu, sk[1], src),
                                      __shfl_sync(0xFFFFFFFFu, sv[0], src), __shfl_sync(0xFFFFFFFFu, sv[1], src));
        const int st = used % NST;
        if (lane == 0) {
          uint8_t* dst = stages + st * LY::STAGE;
          metas[st] = mt;
          if (a.pv.P == 16) {
            mbar_arrive_expect_tx(&bars[st], (uint32_t)((p0 >= 0) + (p1 >= 0)) * 2 * 16 * D);
            if (p0 >= 0) {
              const int y = (int)(a.pv.row0 + ((long long)p0 * H + pl.h) * 16);
              tma_load_2d(dst, &tmK, &bars[st], 0, y);
              tma_load_2d(dst + RK * D, &tmV, &bars[st], 0, y);
            }
            if (p1 >= 0) {
              const int y = (int)(a.pv.row0 + ((long long)p1 * H + pl.h) * 16);
              tma_load_2d(dst + 16 * D, &tmK, &bars[st], 0, y);
              tma_load_2d(dst + RK * D + 16 * D, &tmV, &bars[st], 0, y);
            }
          } else {
            const int y = (int)(a.pv.row0 + (((long long)p0 * H + pl.h) << a.pv.p_shift)) + ((k * RK) & (a.pv.P - 1));
            mbar_arrive_expect_tx(&bars[st], LY::STAGE);
            tma_load_2d(dst, &tmK, &bars[st], 0, y);
            tma_load_2d(dst + RK * D, &tmV, &bars[st], 0, y);
          }
        }
        ++used;
      };
      // ---------------------------------------------------------- keys
      const int first = used;
      int issued = k0;
      while (issued < k1 && issued < k0 + NST) issue(issued++);
      bool alive = true;
      for (int k = k0; k < k1; ++k) {
        const int n = first + (k - k0);
        const int st = n % NST;
        if (!warp_wait(&bars[st], (n / NST) & 1, abort_flag)) {
          alive = false;
          break;
        }
        __syncwarp();
        const uint8_t* kc = stages + st * LY::STAGE;
        const uint8_t* vc = kc + RK * D;
        const float4 mt = metas[st];
        float c[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.0f;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            const uint4 w = *reinterpret_cast<const uint4*>(kc + code_chunk<D>(j * 8 + key_row(g), q * 4 + t4));
            mma_16816(c[j], qa[q * 4 + 0], widen_lo(w.x), widen_hi(w.x));
            mma_16816(c[j], qa[q * 4 + 1], widen_lo(w.y), widen_hi(w.y));
            mma_16816(c[j], qa[q * 4 + 2], widen_lo(w.z), widen_hi(w.z));
            mma_16816(c[j], qa[q * 4 + 3], widen_lo(w.w), widen_hi(w.w));
          }
        }
        // y of row g (and, e = 1, g + 8); columns 2 t4, 2 t4 + 1 of group j
        const float sk1 = a.pv.P == 16 ? mt.y : mt.x, sv1 = a.pv.P == 16 ? mt.w : mt.z;
        const float off0 = __log2f(mt.z), off1 = __log2f(sv1);
        const int key0 = k * RK;
        bool cut = false;
#pragma unroll
        for (int e = 0; e < E; ++e) cut = cut || key0 + RK > hi[e] || key0 < lo[e];
        float mx[E];
        bool raise = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          mx[e] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float s = SPLIT ? c[j][i] + c[j][2 + i] : c[j][2 * e + i];
              float y = fmaf(s, rf[e] * (j < 2 ? mt.x : sk1), j < 2 ? off0 : off1);
              if (cut) {
                const int key = key0 + j * 8 + key_row(2 * t4 + i);
                if (key >= hi[e] || key < lo[e] || key >= pl.t.hi) y = -INFINITY;
              }
              c[j][2 * e + i] = y;
              mx[e] = fmaxf(mx[e], y);
            }
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], 2));
          raise = raise || mx[e] > m[e];
        }
        if (__any_sync(0xFFFFFFFFu, raise)) {
          float al[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float mn = fmaxf(m[e], mx[e]);
            al[e] = mn > m[e] ? ex2f(m[e] - mn) : 1.0f;      // 0 for the first keys of a row
            m[e] = mn;
            l[e] *= al[e];
          }
#pragma unroll
          for (int i = 0; i < DG; ++i) {
            o[i][0] *= al[0];
            o[i][1] *= al[0];
            o[i][2] *= al[E - 1];
            o[i][3] *= al[E - 1];
          }
        }
        uint32_t pa[2][4];
        const float iv0 = 1.0f / mt.z, iv1 = 1.0f / sv1;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float sub = m[e] == -INFINITY ? 0.0f : 8.0f - m[e];
          float ls[2] = {0.0f, 0.0f};                    // of either page
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float w0 = ex2f(c[j][2 * e] + sub), w1 = ex2f(c[j][2 * e + 1] + sub);
            ls[j >> 1] += w0 + w1;
            const uint32_t w = cvt_f16x2(w0, w1);
            pa[j >> 1][(j & 1) * 2 + e] = w;
            if constexpr (SPLIT) {
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w));
              pa[j >> 1][(j & 1) * 2 + 1] = cvt_f16x2(w0 - y.x, w1 - y.y);
            }
          }
          l[e] += ls[0] * iv0 + ls[1] * iv1;
        }
        // O += P V: k pairs are keys (row(2 t4), row(2 t4 + 1)) of groups 2 kk and 2 kk + 1
        const bool edge = key0 + RK > pl.t.hi || key0 < pl.t.lo;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          uint32_t w[4][D / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int kr = kk * 16 + (r >> 1) * 8 + key_row(2 * t4 + (r & 1));
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
            // rows no query sees may hold anything, NaN codes too
            if (edge && (key0 + kr >= pl.t.hi || key0 + kr < pl.t.lo)) {
#pragma unroll
              for (int i = 0; i < D / 32; ++i) w[r][i] = 0u;
            }
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t a01 = __byte_perm(w[0][i], w[1][i], 0x5140), a23 = __byte_perm(w[0][i], w[1][i], 0x7362);
            const uint32_t b01 = __byte_perm(w[2][i], w[3][i], 0x5140), b23 = __byte_perm(w[2][i], w[3][i], 0x7362);
            mma_16816(o[4 * i + 0], pa[kk], widen_lo(a01), widen_lo(b01));
            mma_16816(o[4 * i + 1], pa[kk], widen_hi(a01), widen_hi(b01));
            mma_16816(o[4 * i + 2], pa[kk], widen_lo(a23), widen_lo(b23));
            mma_16816(o[4 * i + 3], pa[kk], widen_hi(a23), widen_hi(b23));
          }
        }
        __syncwarp();                                    // every lane is done with the stage
        if (issued < k1) issue(issued++);
      }
      if (!alive) {
        // copies still in flight land in this block's shared memory: wait (bounded)
        for (int n = first; n < used; ++n)
          if (n >= used - NST) mbar_wait(&bars[n % NST], (n / NST) & 1, nullptr, 100000000ull);
        break;
      }
      // ---------------------------------------------------------- results
#pragma unroll
      for (int e = 0; e < E; ++e) {
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 1);
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 2);
      }
      if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < DG; ++i) {
          o[i][0] += o[i][2];
          o[i][1] += o[i][3];
        }
      }
      const int slot = 2 * worker + (u == pl.at ? 1 : 0);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = pl.tile * RT + g + 8 * e;
        if (r >= rows) continue;
        if (whole) {
          const int i = r / G;
          const float inv = l[e] > 0.0f ? 1.0f / l[e] : 0.0f;
          T* dst = static_cast<T*>(a.out) + (pl.s.s0 + i) * a.out_stride + (size_t)(pl.h * G + r - i * G) * D;
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            uint4* at = reinterpret_cast<uint4*>(dst + (2 * t4 + f) * DG);
#pragma unroll
            for (int c = 0; c < DG / 8; ++c)
              at[c] = make_uint4(pack2<T>(o[8 * c][2 * e + f] * inv, o[8 * c + 1][2 * e + f] * inv),
                                 pack2<T>(o[8 * c + 2][2 * e + f] * inv, o[8 * c + 3][2 * e + f] * inv),
                                 pack2<T>(o[8 * c + 4][2 * e + f] * inv, o[8 * c + 5][2 * e + f] * inv),
                                 pack2<T>(o[8 * c + 6][2 * e + f] * inv, o[8 * c + 7][2 * e + f] * inv));
          }
        } else {
          const size_t at_row = (size_t)slot * RT + g + 8 * e;
          float* dst = a.rows.o + at_row * D;
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int c = 0; c < DG / 4; ++c)
              reinterpret_cast<float4*>(dst + (2 * t4 + f) * DG)[c] =
                  make_float4(o[4 * c][2 * e + f], o[4 * c + 1][2 * e + f], o[4 * c + 2][2 * e + f], o[4 * c + 3][2 * e + f]);
          if (t4 == 0) a.rows.ml[at_row] = make_float2(m[e], l[e]);
        }
      }
      if (u == pl.at && end < item_end) rec = {pl.b, pl.h, pl.tile, (int)((item_end - 1) / stretch)};
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
template <int D, typename T>
static cudaError_t prepare_t() {
  return cudaFuncSetAttribute(paged_attend_rows_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsLayout<D>::ALLOC);
}

cudaError_t prepare_paged_rows(int D) {
  const cudaError_t e = D == 128 ? prepare_t<128, __half>() : prepare_t<64, __half>();
  if (e != cudaSuccess) return e;
  return D == 128 ? prepare_t<128, __nv_bfloat16>() : prepare_t<64, __nv_bfloat16>();
}

template <int D, typename T>
static cudaError_t rows_t(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, int blocks,
                          cudaStream_t st) {
  return launch_pdl(paged_attend_rows_kernel<D, T>, dim3(blocks), dim3(RTHREADS), RowsLayout<D>::ALLOC, st, tmK, tmV, a);
}

cudaError_t launch_paged_rows(const PagedAttn& a, const CUtensorMap& tmK, const CUtensorMap& tmV, bool f16, int blocks,
                              cudaStream_t st) {
  if (a.pv.D == 64)
    return f16 ? rows_t<64, __half>(a, tmK, tmV, blocks, st) : rows_t<64, __nv_bfloat16>(a, tmK, tmV, blocks, st);
  return f16 ? rows_t<128, __half>(a, tmK, tmV, blocks, st) : rows_t<128, __nv_bfloat16>(a, tmK, tmV, blocks, st);
}

}  // namespace kvring_dev
