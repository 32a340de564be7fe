// How the paged attention kernels share their work.
//
// An item is (sequence, key head, tile of TR query rows); its work is the
// tiles of KT keys that any of its rows sees.  All items of a call are laid
// end to end, and every worker takes an equal stretch of that line, so ragged
// lengths and a single long sequence load the GPU alike; an item cut by the
// ends of stretches leaves partial results that a second kernel joins.  The
// lengths are read on the device: a captured call follows them.
//
// Where a kernel's items cost much beside their tiles (FIX > 0), a cut is worth
// avoiding: with fewer items than workers, every item gets the same number of
// workers to itself (one, if there are no more), as if all were as long as the
// longest, unless that makes a stretch longer than the equal one by more than a
// cut costs (kCut).
#pragma once
#include "paged.h"

namespace kvring_dev {

// a / b, both >= 0 (b > 0): 32-bit numbers nearly always, whose division is several times shorter
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

struct Tiles {
  int lo, hi;          // keys that some row of the item sees: [lo, hi), empty when hi <= lo
  int t0, t1;          // tiles of KT keys that hold them
};

template <int TR, int KT>
__device__ __forceinline__ Tiles item_tiles(const PagedAttn& a, const SeqInfo& s, int tile) {
  const int g = a.pv.G;
  int i0 = 0, i1 = s.n - 1;
  if (s.n * g > TR) {
    i0 = tile * TR / g;
    i1 = min(s.n, (tile * TR + TR + g - 1) / g) - 1;
  }
  Tiles t;
  t.hi = a.causal ? max(0, s.len - s.n + i1 + 1) : s.len;
  t.lo = a.window > 0 ? max(0, s.len - s.n + i0 - a.window + 1) : 0;
  const bool any = t.hi > t.lo;
  t.t0 = any ? t.lo / KT : 0;
  t.t1 = any ? (t.hi + KT - 1) / KT : 0;
  return t;
}

// How long every item counts (0: as long as it is), and a worker's stretch then.
struct Cut {
  int pad, stretch;
};

// One kernel's share of the sequences: those with rows in (MIN, MAX].  FIX:
// what an item costs beside its tiles, in tiles.
template <int TR, int KT, int FIX, int MIN, int MAX>
struct Share {
  // pad: 0, or what every item counts
  static __device__ __forceinline__ int units(const Tiles& t, int pad) {
    return pad ? pad : max(t.t1 - t.t0, FIX ? 0 : 1) + FIX;
  }

  // tiles of rows of sequence s that this kernel works on
  static __device__ __forceinline__ int row_tiles(const PagedAttn& a, const SeqInfo& s) {
    const long long rows = (long long)s.n * a.pv.G;
    if (rows <= MIN || rows > MAX || s.n > a.max_new) return 0;
    return (int)((rows + TR - 1) / TR);
  }

  // pre[b] = units of one key head of the sequences before b, pre[n_seqs] the
  // total; all threads of the block.  warp_sums: one entry per warp.  With
  // FIX > 0 (``sums``: three zeros at first, shared): may set pad and a stretch.
  template <int NT>
  static __device__ Cut prefix(const PagedAttn& a, long long* pre, long long* warp_sums, bool report,
                               unsigned long long* sums = nullptr, int workers = 0) {
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
        int most = 0;
        for (int t = 0; t < nt; ++t) {
          const int n = units(item_tiles<TR, KT>(a, s, t), 0);
          u += n;
          most = max(most, n);
        }
        if (FIX > 0 && nt > 0) add_items(sums, u, nt, most);
      } else {
        u = -1;
      }
      pre[b + 1] = u;
    }
    // (with an entry for each thread, a thread scans its own)
    if (MAX > kAlone * TR || B > NT) __syncthreads();
    if constexpr (MAX > kAlone * TR) {
      for (int b = warp; b < B; b += NT / 32) {
        if (pre[b + 1] >= 0) continue;
        bool ok;
        const SeqInfo s = seq_info(a.pb, a.pv.p_shift, b, ok);
        const int nt = row_tiles(a, s);
        long long u = 0;
        int most = 0;
        for (int t = lane; t < nt; t += 32) {
          const int n = units(item_tiles<TR, KT>(a, s, t), 0);
          u += n;
          most = max(most, n);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, off);
        if (FIX > 0) most = __reduce_max_sync(0xFFFFFFFFu, most);
        __syncwarp();
        if (lane == 0) {
          pre[b + 1] = u;
          if (FIX > 0) add_items(sums, u, nt, most);
        }
      }
      __syncthreads();
    }
    Cut cut = {0, 0};
    if constexpr (FIX > 0) {
      const long long total = (long long)sums[0] * a.pv.H, items = (long long)sums[1] * a.pv.H;
      const int most = (int)sums[2];
      if (items > 0 && items <= workers) {
        const int per = workers / (int)items;            // workers of an item
        const int part = max((most + per - 1) / per, kLeast);
        if (part <= max(quotient(total + workers - 1, workers), (long long)kLeast) + kCut)
          cut = {(most + part - 1) / part * part, part};
      }
      if (cut.pad) {
        for (int b = tid; b < B; b += NT) {
          bool ok;
          pre[b + 1] = (long long)row_tiles(a, seq_info(a.pb, a.pv.p_shift, b, ok)) * cut.pad;
        }
        __syncthreads();
      }
    }
    // inclusive scan: each thread a run of entries (at most one, nearly always), then the runs' sums
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
    return cut;
  }

  // units, items, and the longest item
  static __device__ __forceinline__ void add_items(unsigned long long* sums, long long u, int items, int most) {
    atomicAdd(&sums[0], (unsigned long long)u);
    atomicAdd(&sums[1], (unsigned long long)items);
    atomicMax(&sums[2], (unsigned long long)most);
  }

  // Units of a stretch, at least (64 tokens over 4,000, 8 key heads: 38.5 us;
  // with 6: 41.5, with 9: 44.4), and what a cut costs: a second piece's
  // queries, fp32 results and their joining (1,100 tokens over 4,000: 100.4 us;
  // with 4, which cuts there: 107.8; with 12, which does not cut 512 tokens
  // over 16,000: 152.7 instead of 140.7).  Items to themselves take 22.9 us for
  // a prompt of 128 and 38 us for one of 1,024, cut ones 31.6 and 47.
  static constexpr int kLeast = 4;
  static constexpr int kCut = 8;
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
__device__ Place find_place(const PagedAttn& a, const long long* pre, long long u, int pad = 0) {
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
  p.h = per_head > 0 ? (int)quotient(rest, per_head) : 0;
  rest -= p.h * per_head;
  p.at = u - rest;
  p.tile = 0;
  for (int t0 = 0; t0 < p.row_tiles; t0 += 32) {
    const int t = t0 + lane;
    const int n = t < p.row_tiles ? SH::units(item_tiles<TR, KT>(a, p.s, t), pad) : 0;
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
  p.units = SH::units(p.t, pad);
  return p;
}

// The next item; false at the end of the line.
template <class SH, int TR, int KT>
__device__ __forceinline__ bool next_place(const PagedAttn& a, Place& p, int pad = 0) {
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
  p.units = SH::units(p.t, pad);
  return true;
}

}  // namespace kvring_dev
