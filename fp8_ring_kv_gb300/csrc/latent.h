// Internal definitions of the latent cache: the calls' arguments and the
// kernels' host-side entry points.
//
// The paged cache's view, batch and sharing of work serve here as well: one
// "key head" (the row that all heads share) with all query heads on it in the
// absorbed form, and a key head per query head in the expanded form.
#pragma once
#include "paged.h"

namespace kvring_dev {

constexpr int kLatRope = 64;               // numbers of the rotated part
constexpr int kLatHead = 128;              // of a head's key part and value in the expanded form
constexpr int kLatMax = 512;               // of a latent, at most
constexpr float kLatMinScale = 0x1p-40f;   // a row's scale, at least
constexpr float kLatMaxScale = 0x1p40f;    // and at most (a row beyond is marked)
constexpr int kLatRows = 64;               // query rows of an item of the absorbed form, at most

struct Strides {
  long long token, head;
};

// One absorbed call.  a.pv: k_codes, k_scale the cache's, D = C; a.q: q_latent.
// a.tiles: pieces of [kLatRows][C].
struct LatentAttn {
  PagedAttn a;
  const void* q_rope;
  Strides q, qr, o;
  int32_t code_rows;               // of all layers: the code arrays' height
};

// One expanded call.  a.pv.H heads with G = 1; a.pb.table = kv_start, a
// "page" of 2^22 keys per sequence.  a.tiles: pieces of [kTilesRows][128].
struct ExpandedAttn {
  PagedAttn a;
  Strides q, o;
  const void* v;
  long long v_token, v_head;
  int32_t n_keys;
};

// mbar_wait and warp_wait in fewer instructions: these kernels wait in many
// places, and their roles' loops share the instruction caches.  The limit counts
// tests, of some tens of cycles to a microsecond each (a third of a second at least).
constexpr uint32_t kWaitTests = 1u << 24;
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  for (uint32_t tests = 1; !mbar_try_wait(bar, parity); ++tests)
    if ((tests & 255u) == 0) {
      if (tests >= kWaitTests) *abort = 1;
      if (*abort) return false;
    }
  return true;
}
__device__ __forceinline__ bool bar_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort));
}

size_t latent_scratch_bytes(int C);
// pieces of ``rows`` rows of ``width`` numbers
void latent_carve_scratch(uint8_t* base, int rows, int width, PagedAttn* a);

cudaError_t launch_latent_append(const PagedView& pv, const PagedBatch& pb, const void* latent, long long latent_stride,
                                 const void* rope, long long rope_stride, const int32_t* pos, bool f16, cudaStream_t st);
cudaError_t launch_latent_read(const PagedView& pv, const PagedBatch& pb, void* out, long long out_stride, bool f16,
                               cudaStream_t st);
cudaError_t prepare_latent_attend();
// tmC: the code rows as [rows][W] u8, box {128, P}, 128-byte swizzle; tmR: box {64, P}, 64-byte swizzle
cudaError_t launch_latent_attend(const LatentAttn& la, const CUtensorMap& tmC, const CUtensorMap& tmR, bool f16, int sms,
                                 cudaStream_t st);

// the items that several blocks share: pieces of up to ``rows`` rows of a.pv.D
// numbers, ``slot_rows`` rows of room each
cudaError_t launch_latent_join(const PagedAttn& a, const Strides& o, int slot_rows, int rows, bool f16, int blocks,
                               cudaStream_t st);
cudaError_t prepare_latent_expanded();
// tmK, tmV: [heads][keys][128] in 16 bits, boxes {64, 128, 1} and {64, 64, 1}; tmR: [keys][64], box {64, 128}
cudaError_t launch_latent_expanded(const ExpandedAttn& xa, const CUtensorMap& tmK, const CUtensorMap& tmR,
                                   const CUtensorMap& tmV, bool f16, int sms, cudaStream_t st);

}  // namespace kvring_dev
