// How the paged attention kernels share their work.
//
// An item is (sequence, key head, tile of TR query rows); its work is the
// tiles of KT keys that any of its rows sees.  All items of a call are laid
// end to end, and every worker takes an equal stretch of that line, so ragged
// lengths and a single long sequence load the GPU alike; an item cut by the
// ends of stretches leaves partial results that a second kernel joins.  The
// lengths are read on the device: a captured call follows them.
#pragma once
#include "paged.h"

namespace kvring_dev {

struct Tiles {
  int lo, hi;          // keys that some row of the item sees: [lo, hi), empty when hi <= lo
  int t0, t1;          // tiles of KT keys that hold them
};

template <int TR, int KT>
__device__ __forceinline__ Tiles item_tiles(const PagedAttn& a, const SeqInfo& s, int tile) {
  const int g = a.pv.G;
  const int i0 = tile * TR / g;
  const int i1 = min(s.n, (tile * TR + TR + g - 1) / g) - 1;
  Tiles t;
  t.hi = a.causal ? max(0, s.len - s.n + i1 + 1) : s.len;
  t.lo = a.window > 0 ? max(0, s.len - s.n + i0 - a.window + 1) : 0;
  const bool any = t.hi > t.lo;
  t.t0 = any ? t.lo / KT : 0;
  t.t1 = any ? (t.hi + KT - 1) / KT : 0;
  return t;
}

// One kernel's share of the sequences: those with rows in (MIN, MAX].  FIX:
// what an item costs beside its tiles, in tiles.
template <int TR, int KT, int FIX, int MIN, int MAX>
struct Share {
  static __device__ __forceinline__ int units(const Tiles& t) { return max(t.t1 - t.t0, FIX ? 0 : 1) + FIX; }

  // tiles of rows of sequence s that this kernel works on
  static __device__ __forceinline__ int row_tiles(const PagedAttn& a, const SeqInfo& s) {
    const long long rows = (long long)s.n * a.pv.G;
    if (rows <= MIN || rows > MAX || s.n > a.max_new) return 0;
    return (int)((rows + TR - 1) / TR);
  }

  // pre[b] = units of one key head of the sequences before b, pre[n_seqs] the
  // total; all threads of the block.  warp_sums: one entry per warp.
  template <int NT>
  static __device__ void prefix(const PagedAttn& a, long long* pre, long long* warp_sums, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.pb.n_seqs;
    constexpr int kAlone = 4;            // row tiles that one thread sums by itself
    for (int b = tid; b < B; b += NT) {
      bool ok;
      const SeqInfo s = seq_info(a.pb, a.pv.p_shift, b, ok);
      if (report && (!ok || s.n > a.max_new)) atomicOr(&a.pv.state[PST_ERR], DEVERR_SEQ);
      const int nt = row_tiles(a, s);
      long long u = 0;
      if (nt <= kAlone) {
        for (int t = 0; t < nt; ++t) u += units(item_tiles<TR, KT>(a, s, t));
      } else {
        u = -1;
      }
      pre[b + 1] = u;
    }
    __syncthreads();
    for (int b = warp; b < B; b += NT / 32) {
      if (pre[b + 1] >= 0) continue;
      bool ok;
      const SeqInfo s = seq_info(a.pb, a.pv.p_shift, b, ok);
      const int nt = row_tiles(a, s);
      long long u = 0;
      for (int t = lane; t < nt; t += 32) u += units(item_tiles<TR, KT>(a, s, t));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, off);
      __syncwarp();
      if (lane == 0) pre[b + 1] = u;
    }
    __syncthreads();
    // inclusive scan: each thread a run of entries, then the runs' sums
    const int run = (B + NT - 1) / NT;
    const int b0 = min(B, tid * run), b1 = min(B, b0 + run);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += pre[b + 1];
    long long inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
      if (lane >= off) inc += o;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    long long base = inc - sum;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    for (int b = b0; b < b1; ++b) {
      base += pre[b + 1];
      pre[b + 1] = base;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
  }
};

// A place on the line of items: (sequence, key head, row tile), the unit at
// which that item begins, and its numbers.
struct Place {
  int b, h, tile;
  long long at;
  SeqInfo s;
  Tiles t;
  int units, row_tiles;
};

// The item that holds unit u (0 <= u < H * pre[n_seqs]); one warp.
template <class SH, int TR, int KT>
__device__ Place find_place(const PagedAttn& a, const long long* pre, long long u) {
  const int lane = threadIdx.x & 31;
  const int H = a.pv.H;
  int lo = 0, hi = a.pb.n_seqs - 1;      // the last b with pre[b] * H <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] * H <= u) lo = mid; else hi = mid - 1;
  }
  Place p;
  p.b = lo;
  bool ok;
  p.s = seq_info(a.pb, a.pv.p_shift, lo, ok);
  p.row_tiles = SH::row_tiles(a, p.s);
  const long long per_head = pre[lo + 1] - pre[lo];
  long long rest = u - pre[lo] * H;
  p.h = per_head > 0 ? (int)(rest / per_head) : 0;
  rest -= p.h * per_head;
  p.at = u - rest;
  p.tile = 0;
  for (int t0 = 0; t0 < p.row_tiles; t0 += 32) {
    const int t = t0 + lane;
    const int n = t < p.row_tiles ? SH::units(item_tiles<TR, KT>(a, p.s, t)) : 0;
    long long inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
      if (lane >= off) inc += o;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, inc > rest);
    if (past) {
      const int l = __ffs(past) - 1;
      p.tile = t0 + l;
      const long long before = __shfl_sync(0xFFFFFFFFu, inc - n, l);
      p.at += before;
      break;
    }
    const long long all = __shfl_sync(0xFFFFFFFFu, inc, 31);
    rest -= all;
    p.at += all;
  }
  p.t = item_tiles<TR, KT>(a, p.s, p.tile);
  p.units = SH::units(p.t);
  return p;
}

// The next item; false at the end of the line.
template <class SH, int TR, int KT>
__device__ __forceinline__ bool next_place(const PagedAttn& a, Place& p) {
  p.at += p.units;
  if (++p.tile >= p.row_tiles) {
    p.tile = 0;
    if (++p.h >= a.pv.H) {
      p.h = 0;
      do {
        if (++p.b >= a.pb.n_seqs) return false;
        bool ok;
        p.s = seq_info(a.pb, a.pv.p_shift, p.b, ok);
        p.row_tiles = SH::row_tiles(a, p.s);
      } while (p.row_tiles == 0);
    }
  }
  p.t = item_tiles<TR, KT>(a, p.s, p.tile);
  p.units = SH::units(p.t);
  return true;
}

}  // namespace kvring_dev
