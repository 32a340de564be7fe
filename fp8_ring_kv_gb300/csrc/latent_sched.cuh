// The line of items of a call of few short sequences, by one warp.
//
// Share::prefix works with a whole block: five barriers and its code, 4 us of a
// call that decodes a token.  Up to 32 sequences of a few row tiles each are a lane
// each here.
#pragma once
#include "latent.h"
#include "paged_sched.cuh"

namespace kvring_dev {

constexpr int kLaneTiles = 4;                // row tiles that a lane sums

struct LineOfWork {
  Cut cut;
  int small;                                 // whether it was done here
};

// Share::prefix, by all threads; ``line`` in shared memory (warp_sums, sums as
// there).  The same numbers, whichever way they come.
template <class SH, int TR, int KT, int NT>
__device__ __forceinline__ Cut latent_prefix(const PagedAttn& a, long long* pre, long long* warp_sums, bool report,
                                             unsigned long long* sums, int workers, LineOfWork* line) {
  const int lane = threadIdx.x & 31, B = a.pb.n_seqs;
  if (B <= 32) {
    if (threadIdx.x < 32) {
      bool ok = true;
      SeqInfo s = {0, 0, 0};
      if (lane < B) s = seq_info(a.pb, a.pv.p_shift, lane, ok);
      const int nt = lane < B ? SH::row_tiles(a, s) : 0;
      const bool small = __all_sync(0xFFFFFFFFu, nt <= kLaneTiles);
      if (small) {
        if (report && (!ok || s.n > a.max_new)) atomicOr(&a.pv.state[PST_ERR], DEVERR_SEQ);
        int u = 0, most = 0;
        for (int t = 0; t < nt; ++t) {
          const int n = SH::units(item_tiles<TR, KT>(a, s, t), 0);
          u += n;
          most = max(most, n);
        }
        // (a sequence has at most 2^22 / KT tiles of keys: 32-bit sums)
        const long long total = (long long)__reduce_add_sync(0xFFFFFFFFu, u) * a.pv.H;
        const int items = __reduce_add_sync(0xFFFFFFFFu, nt) * a.pv.H;
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        const Cut cut = SH::choose(total, items, most, workers);
        long long inc = cut.pad ? (long long)nt * cut.pad : u;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, off);
          if (lane >= off) inc += o;
        }
        if (lane < B) pre[lane + 1] = inc;
        if (lane == 0) {
          pre[0] = 0;
          line->cut = cut;
        }
      }
      if (lane == 0) line->small = small;
    }
    __syncthreads();
    if (line->small) return line->cut;
  }
  return SH::template prefix<NT>(a, pre, warp_sums, report, sums, workers);
}

}  // namespace kvring_dev
