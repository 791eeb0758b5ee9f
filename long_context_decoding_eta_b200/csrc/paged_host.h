// Host-side helpers of the paged-cache entry points: checks of the pool's size and the
// layout of the bookkeeping array `state`.
#pragma once

#include <math.h>

#include "eta_host.h"

namespace eta {

// Word offsets of the sections of `state` (each padded to 4 words, 16 bytes).
struct PageLayout {
  size_t header, lengths, table, ref, free_list, words;
};

inline PageLayout page_layout(const eta_dims_t* d, int32_t n_pages) {
  PageLayout L;
  size_t x = 0;
  L.header = x;    x = align_up(x + 8, 4);
  L.lengths = x;   x = align_up(x + (size_t)d->B, 4);
  L.table = x;     x = align_up(x + (size_t)d->B * num_blocks(d), 4);
  L.ref = x;       x = align_up(x + (size_t)n_pages, 4);
  L.free_list = x; x = align_up(x + (size_t)n_pages, 4);
  L.words = x;
  return L;
}

// Dims and pool size of a paged call.  TMA row coordinates (page, head, token) are
// 32-bit, which bounds the pool.
inline eta_status_t check_pool(const eta_dims_t* d, int32_t n_pages) {
  const eta_status_t st = check_dims(d);
  if (st != ETA_OK) return st;
  if (n_pages <= 0) return ETA_ERR_INVALID_ARG;
  if ((uint64_t)n_pages * d->Hkv * d->blk >= (1ull << 31)) return ETA_ERR_UNSUPPORTED;
  return ETA_OK;
}

// 1 / T of a soft gate, finite (and so 0 times it is 0) where T is too small for that.
inline float inverse_temperature(float T) { return fminf(1.f / T, 2e38f); }

}  // namespace eta
