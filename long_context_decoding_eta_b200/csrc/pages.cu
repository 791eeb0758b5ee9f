// Bookkeeping and data movement of a paged KV cache: append, fork, free, compact, copy
// (include/eta.h, "Paged caches").  No counterpart in the ETA pages.
//
// A call decides everything from the state before it, then carries it out.  Page numbers
// come from prefix sums and bitmaps, never from the arrival order of atomics, so the same
// calls always give the same tables; the only atomics are integer counts whose order does
// not matter.  The data kernels move whole 16-byte vectors and are bound by HBM (read +
// write of the moved tokens), the bookkeeping by launch latency.  So append, fork and free
// are one launch each: every CTA works the whole decision out for itself (a scan over the
// rows or pairs), and what it was read from, the lengths and the free count, is written by
// the CTA that finishes last.  Above 1,024 rows, or 64 forked pairs, a plan kernel of one
// CTA decides for all.  Measured (us a launch, replayed): append of 64 rows, 11,000 tokens of
// 2 KB, 9.9 (read + write 4.6 TB/s); free and fork of 6 rows 6.5 and 5.4, of 56 rows of 300 pages 11.5 and
// 7.7; compaction of 2.06 GB 333 (6.2 TB/s), of 34 MB 13; 1,777 pages of 128 KB 79 (5.9 TB/s).
#include <algorithm>

#include "eta_common.cuh"
#include "paged_host.h"

namespace eta {
namespace pg {

constexpr int kPlan = 1024;       // threads of a one-CTA plan
constexpr int kCopy = 256;        // threads of a data-moving CTA
// Up to kLocal rows every CTA of an append plans by itself (us: 64 rows 5.2, with a plan launch
// 7.2; 512 rows 6.8 and 7.8; 1,024 rows 8.2 and 8.6), up to kLocalPairs pairs every CTA of a fork,
// of which there are 8 a pair (4 pairs 5.4 and 6.2; 64 pairs 6.4 and 6.4; 96 pairs 6.8 and 6.4;
// 256 pairs 14.2 and 7.6).
constexpr int kLocal = 1024;
constexpr int kLocalPairs = 64;
constexpr int kChunk = 4096;      // pages per CTA of the compaction's scan
// Up to kOwnCount chunks every CTA of the scan counts all of the pool by itself.  A compaction
// is then two launches instead of three, 12.3 us of the host's time instead of 14.0, for 0.2
// to 0.6 us more of the GPU's (1,024 pages with nothing to move 8.0 us, with a count launch 7.6;
// 16,384 pages 8.2 and 7.6; 32,768 pages 8.4 and 8.0, and 50.4 and 50.5 moving a quarter).
constexpr int kOwnCount = 8;
// Copies of at most kOwnCheck pairs and kOwnBytes, read and written once, are checked by every
// copying CTA by itself (us: 2,048 pairs of 16 KB, K and V, 11.8, with a plan launch 15.6; 1,024
// pairs of 128 KB 46.9 and 47.0; 1,777 of them 84.4 and 78.5; 2,048 of them 95.3 and 89.1).
constexpr int kOwnCheck = 2048;
constexpr int64_t kOwnBytes = 1 << 27;

struct Pool {
  int B, NB, n_pages, Hkv, blk, d;
  int32_t *header, *lengths, *table, *ref, *free_list;
  eta_bf16_t *K, *V;
  int32_t* status;
};

// Exclusive prefix sum of v over the NT threads of the CTA; total is the sum.
template <int NT>
ETA_DEV int block_scan(int v, int* wsum, int& total) {
  constexpr int NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int x = wsum[w];
    if (w < warp) before += x;
    sum += x;
  }
  total = sum;
  __syncthreads();
  return before + incl - v;
}

// True in every thread of the CTA that gets here last of the grid; `done` counts them and
// is left at zero.  What the other CTAs wrote before is visible to it.
ETA_DEV bool last_cta(int32_t* done, int ctas) {
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int last = atomicAdd(done, 1) == ctas - 1;
    if (last) *done = 0;
    s_last = last;
  }
  __syncthreads();
  __threadfence();
  return s_last;
}

ETA_DEV int blocks_of(int n, int blk) { return (n + blk - 1) / blk; }

ETA_DEV bool page_ok(const Pool& p, int page) { return page >= 0 && page < p.n_pages; }

// ------------------------------------------------------------------------------- init
__global__ void __launch_bounds__(kCopy) init_kernel(const Pool p) {
  ETA_PDL_ENTRY();
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long t0 = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  for (long long i = t0; i < (long long)p.B * p.NB; i += step) p.table[i] = -1;
  for (long long i = t0; i < p.B; i += step) p.lengths[i] = 0;
  for (long long i = t0; i < p.n_pages; i += step) {
    p.ref[i] = 0;
    p.free_list[i] = p.n_pages - 1 - (int)i;
  }
  if (t0 < 8) p.header[t0] = t0 == 0 ? p.n_pages : 0;
}

// ----------------------------------------------------------------------------- append
// Per row, rec[b]: the length before the call (-1: refused, or nothing to do) and how many
// pages the rows before it take.  Returns {free pages before the call, pages taken};
// {.., -1}: the offsets are out of order and nothing is appended.
template <int NT>
ETA_DEV int2 append_plan(const Pool& p, const int32_t* cu, int n_new, int2* rec,
                         int32_t* status) {
  __shared__ int wsum[NT / 32];
  __shared__ int s_used;
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  if (threadIdx.x == 0) s_used = 0;
  bool bad = false;
  for (int b = threadIdx.x; b < p.B; b += NT)
    bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > n_new;
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_status(status, ETA_DEVSTAT_BAD_LENGTH);
    return make_int2(n_free, -1);
  }
  int carry = 0;
  for (int base = 0; base < p.B; base += NT) {
    const int b = base + threadIdx.x;
    int need = 0, len = 0;
    bool ok = false;
    if (b < p.B) {
      const int n = cu[b + 1] - cu[b];
      len = p.lengths[b];
      if (len < 0 || len > p.NB * p.blk || n > p.NB * p.blk - len) {
        set_status(status, ETA_DEVSTAT_BAD_LENGTH);
      } else {
        ok = n > 0;
        if (ok && len % p.blk != 0) {
          const int last = p.table[(size_t)b * p.NB + len / p.blk];
          if (!page_ok(p, last) || p.ref[last] != 1) {
            set_status(status, ETA_DEVSTAT_BAD_ROW);
            ok = false;
          }
        }
        if (ok) need = blocks_of(len + n, p.blk) - blocks_of(len, p.blk);
      }
    }
    int total;
    const int before = carry + block_scan<NT>(need, wsum, total);
    if (need > 0) {
      if (before + need <= n_free) {
        atomicMax(&s_used, before + need);
      } else {
        set_status(status, ETA_DEVSTAT_NO_PAGE);
        ok = false;
      }
    }
    if (b < p.B) rec[b] = make_int2(ok ? len : -1, before);
    carry += total;
  }
  __syncthreads();
  return make_int2(n_free, s_used);
}

// The lengths and the free count after the call.
template <int NT>
ETA_DEV void append_publish(const Pool& p, const int32_t* cu, const int2* rec, int2 f) {
  if (f.y < 0) return;
  for (int b = threadIdx.x; b < p.B; b += NT)
    if (rec[b].x >= 0) p.lengths[b] = rec[b].x + cu[b + 1] - cu[b];
  if (threadIdx.x == 0) p.header[0] = f.x - f.y;
}

__global__ void __launch_bounds__(kPlan)
append_plan_kernel(const Pool p, const int32_t* __restrict__ cu, int n_new, int2* rec) {
  ETA_PDL_ENTRY();
  const int2 f = append_plan<kPlan>(p, cu, n_new, rec, p.status);
  append_publish<kPlan>(p, cu, rec, f);
  if (threadIdx.x == 0) rec[p.B] = f;
}

// One warp per new token: finds its row, its page (from the table, or from the free
// list where the block is new), and writes the token's Hkv key and value vectors.  The
// warp of a new block's first token enters the page into the table.
// LOCAL: the CTA plans by itself; else plan_g is append_plan_kernel's.
template <bool LOCAL>
__global__ void __launch_bounds__(kCopy, 4)
append_kernel(const Pool p, const int32_t* __restrict__ cu_g, int n_new, const int2* plan_g,
              int32_t* done, const uint4* __restrict__ kn, const uint4* __restrict__ vn) {
  ETA_PDL_ENTRY();
  __shared__ int2 s_rec[LOCAL ? kLocal : 1];
  __shared__ int s_cu[LOCAL ? kLocal + 1 : 1];
  const int2* rec = plan_g;
  const int32_t* cu = cu_g;
  int2 f;
  if constexpr (LOCAL) {
    for (int b = threadIdx.x; b <= p.B; b += kCopy) s_cu[b] = cu_g[b];
    __syncthreads();
    f = append_plan<kCopy>(p, s_cu, n_new, s_rec, blockIdx.x == 0 ? p.status : nullptr);
    rec = s_rec;
    cu = s_cu;
  } else {
    f = plan_g[p.B];
  }
  const int lane = threadIdx.x & 31;
  const int vd = p.d / 8, nv = p.Hkv * vd;   // 16-byte vectors of a token's keys
  const int t0 = blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5);
  for (int t = f.y < 0 ? n_new : t0; t < n_new; t += gridDim.x * (kCopy / 32)) {
    int lo = 0, hi = p.B - 1;                // the last row with cu[row] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int b = lo, c0 = cu[b];
    const int2 r = rec[b];
    if (t < c0 || t >= cu[b + 1] || r.x < 0) continue;
    const int pos = r.x + t - c0;
    const int j = pos / p.blk, slot = pos - j * p.blk;
    if (!ETA_IN_BOUNDS(j, p.NB, p.status)) continue;
    const int first_new = blocks_of(r.x, p.blk);
    int page;
    if (j >= first_new) {
      const int k = f.x - 1 - (r.y + j - first_new);
      if (!ETA_IN_BOUNDS(k, p.n_pages, p.status)) continue;
      page = p.free_list[k];
      if (page_ok(p, page) && lane == 0 && slot == 0) {
        p.table[(size_t)b * p.NB + j] = page;
        p.ref[page] = 1;
      }
    } else {
      page = p.table[(size_t)b * p.NB + j];
    }
    if (!page_ok(p, page)) {
      if (lane == 0) set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      continue;
    }
    for (int i = lane; i < nv; i += 32) {
      const int g = i / vd, x = i - g * vd;
      const size_t to = (((size_t)page * p.Hkv + g) * p.blk + slot) * vd + x;
      const uint4 a = kn[(size_t)t * nv + i], c = vn[(size_t)t * nv + i];
      reinterpret_cast<uint4*>(p.K)[to] = a;
      reinterpret_cast<uint4*>(p.V)[to] = c;
    }
  }
  if constexpr (LOCAL)
    if (last_cta(done, gridDim.x)) append_publish<kCopy>(p, s_cu, s_rec, f);
}

// ------------------------------------------------------------------------------- fork
// rec[i]: the source's length (-1: the pair is refused) and the new last page (-1: none).
// first[row]: scratch, the first pair that names the row as its dst.  Returns {free pages
// before the call, pages taken}.
template <int NT>
ETA_DEV int2 fork_plan(const Pool& p, const int32_t* src, const int32_t* dst, int n,
                       int32_t* first, int2* rec, int32_t* status) {
  __shared__ int wsum[NT / 32];
  __shared__ int s_used;
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  if (threadIdx.x == 0) s_used = 0;
  for (int i = threadIdx.x; i < n; i += NT) {
    const int t = dst[i];
    if (t >= 0 && t < p.B) first[t] = 0x7fffffff;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += NT) {
    const int t = dst[i];
    if (t >= 0 && t < p.B) atomicMin(&first[t], i);
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < n; base += NT) {
    const int i = base + threadIdx.x;
    int need = 0, len = -1;
    if (i < n) {
      const int f = src[i], t = dst[i];
      if (f >= 0 && f < p.B && t >= 0 && t < p.B &&
          *reinterpret_cast<volatile int32_t*>(first + t) == i && p.lengths[t] == 0) {
        len = min(max(p.lengths[f], 0), p.NB * p.blk);
        need = len % p.blk != 0;
      } else {
        set_status(status, ETA_DEVSTAT_BAD_ROW);
      }
    }
    int total;
    const int before = carry + block_scan<NT>(need, wsum, total);
    int page = -1;
    if (need) {
      if (before < n_free) {
        page = p.free_list[n_free - 1 - before];
        atomicMax(&s_used, before + 1);
      } else {
        set_status(status, ETA_DEVSTAT_NO_PAGE);
        len = -1;
      }
    }
    if (i < n) rec[i] = make_int2(len, page);
    carry += total;
  }
  __syncthreads();
  return make_int2(n_free, s_used);
}

template <int NT>
ETA_DEV void fork_publish(const Pool& p, const int32_t* dst, int n, const int2* rec, int2 f) {
  for (int i = threadIdx.x; i < n; i += NT)
    if (rec[i].x >= 0) p.lengths[dst[i]] = rec[i].x;
  if (threadIdx.x == 0) p.header[0] = f.x - f.y;
}

__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                 int n, int32_t* first, int2* rec) {
  ETA_PDL_ENTRY();
  const int2 f = fork_plan<kPlan>(p, src, dst, n, first, rec, p.status);
  fork_publish<kPlan>(p, dst, n, rec, f);
}

// Grid (pairs, parts): the parts of a pair share its table row and its last page.
// LOCAL: the CTA plans by itself; else plan_g is fork_plan_kernel's.
template <bool LOCAL>
__global__ void __launch_bounds__(kCopy)
fork_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            int n, const int2* plan_g, int32_t* done) {
  ETA_PDL_ENTRY();
  __shared__ int2 s_rec[LOCAL ? kLocalPairs : 1];
  __shared__ int32_t s_first[LOCAL ? kLocal : 1];      // by row
  const int i = blockIdx.x;
  int2 fr = make_int2(0, 0);
  const int2* rec = plan_g;
  if constexpr (LOCAL) {
    fr = fork_plan<kCopy>(p, src, dst, n, s_first, s_rec,
                          (blockIdx.x | blockIdx.y) == 0 ? p.status : nullptr);
    rec = s_rec;
  }
  const int2 r = rec[i];
  if (r.x >= 0) {
    const int f = src[i], t = dst[i];
    const int full = r.x / p.blk, part = r.x - full * p.blk;
    const int tid = blockIdx.y * kCopy + threadIdx.x, step = gridDim.y * kCopy;
    for (int j = tid; j < full; j += step) {
      const int page = p.table[(size_t)f * p.NB + j];
      p.table[(size_t)t * p.NB + j] = page;
      if (page_ok(p, page)) atomicAdd(&p.ref[page], 1);
      else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
    }
    if (tid == 0 && part && page_ok(p, r.y)) {
      p.table[(size_t)t * p.NB + full] = r.y;
      p.ref[r.y] = 1;
    }
    if (part) {
      const int old = p.table[(size_t)f * p.NB + full];
      if (page_ok(p, old) && page_ok(p, r.y)) {
        const int vd = p.d / 8, per = part * vd;     // 16-byte vectors of one head's tokens
        for (int x = tid; x < p.Hkv * per; x += step) {
          const int g = x / per, y = x - g * per;
          const size_t from = ((size_t)old * p.Hkv + g) * p.blk * vd + y;
          const size_t to = ((size_t)r.y * p.Hkv + g) * p.blk * vd + y;
          const uint4 a = reinterpret_cast<const uint4*>(p.K)[from];
          const uint4 c = reinterpret_cast<const uint4*>(p.V)[from];
          reinterpret_cast<uint4*>(p.K)[to] = a;
          reinterpret_cast<uint4*>(p.V)[to] = c;
        }
      } else if (tid == 0) {
        set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      }
    }
  }
  if constexpr (LOCAL)
    if (last_cta(done, gridDim.x * gridDim.y)) fork_publish<kCopy>(p, dst, n, s_rec, fr);
}

// ------------------------------------------------------------------------------- free
// Grid (rows, parts).  A table entry is taken with an exchange, so a row named twice
// gives its pages back once; a page whose last reference goes is marked in the bitmap.
// The CTA that finishes last pushes the marked pages in descending order, clears the
// bitmap, and empties the rows.
__global__ void __launch_bounds__(kCopy)
free_kernel(const Pool p, const int32_t* __restrict__ rows, int n, uint32_t* bitmap,
            int32_t* done) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[kCopy / 32];
  const int row = rows[blockIdx.x];
  if (row < 0 || row >= p.B) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, ETA_DEVSTAT_BAD_ROW);
  } else {
    const int nb = min(blocks_of(max(p.lengths[row], 0), p.blk), p.NB);
    for (int j = blockIdx.y * kCopy + threadIdx.x; j < nb; j += gridDim.y * kCopy) {
      const int page = atomicExch(&p.table[(size_t)row * p.NB + j], -1);
      if (page == -1) continue;
      if (!page_ok(p, page)) {
        set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
        continue;
      }
      const int old = atomicSub(&p.ref[page], 1);
      if (old == 1) {
        atomicOr(&bitmap[page >> 5], 1u << (page & 31));
      } else if (old <= 0) {
        atomicAdd(&p.ref[page], 1);
        set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      }
    }
  }
  if (!last_cta(done, gridDim.x * gridDim.y)) return;
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  for (int i = threadIdx.x; i < n; i += kCopy) {
    const int b = rows[i];
    if (b >= 0 && b < p.B) p.lengths[b] = 0;
  }
  const int nw = (p.n_pages + 31) / 32;
  int at = n_free;
  for (int base = 0; base < nw; base += kCopy) {      // the highest pages first
    const int w = nw - 1 - (base + (int)threadIdx.x);
    const uint32_t m = w >= 0 ? __ldcg(bitmap + w) : 0u;
    int total;
    const int k = at + block_scan<kCopy>(__popc(m), wsum, total);
    if (m) bitmap[w] = 0u;
    // a warp writes one word's pages after the other, a lane a page: the stores coalesce
    const int lane = threadIdx.x & 31, w0 = nw - 1 - (base + (int)(threadIdx.x & ~31u));
#pragma unroll 4
    for (int u = 0; u < 32; ++u) {
      const uint32_t mu = __shfl_sync(0xffffffffu, m, u);
      const int ku = __shfl_sync(0xffffffffu, k, u) + __popc(mu >> lane >> 1);
      if (!(mu >> lane & 1u)) continue;
      if (ku < p.n_pages) p.free_list[ku] = (w0 - u) * 32 + lane;
      else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
    }
    at += total;
  }
  if (threadIdx.x == 0) p.header[0] = min(at, p.n_pages);
}

// ---------------------------------------------------------------------------- compact
struct Moves {
  int32_t* head;      // [0] pages in use, [1] moves
  int32_t* chunk;     // pages in use of each chunk of kChunk
  int32_t* hole;      // the free numbers below n_live, ascending
  int32_t* mover;     // the pages in use at or above n_live, ascending
  int32_t* rank;      // rank[page] of a mover
};

__global__ void __launch_bounds__(kPlan) compact_count_kernel(const Pool p, const Moves m) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[kPlan / 32];
  int v = 0;
#pragma unroll
  for (int u = 0; u < kChunk / kPlan; ++u) {
    const int i = blockIdx.x * kChunk + u * kPlan + threadIdx.x;
    v += i < p.n_pages && p.ref[i] > 0;
  }
  int total;
  block_scan<kPlan>(v, wsum, total);
  if (threadIdx.x == 0) m.chunk[blockIdx.x] = total;
}

// OWN: a small pool, every CTA counts all of it by itself (no compact_count_kernel).
template <bool OWN>
__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Pool p, const Moves m) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[kPlan / 32];
  __shared__ int4 sums[kPlan / 32];
  const int n_live = p.n_pages - p.header[0];
  int before = 0, below = 0, all = 0;       // live before this chunk, below n_live, in all
  if constexpr (OWN) {
    constexpr int kQ = kOwnCount * kChunk / 4 / kPlan;
    const int nq = (p.n_pages + 3) / 4;     // the section is padded to 4 words
    int4 r[kQ];
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int q = u * kPlan + threadIdx.x;
      r[u] = q < nq ? reinterpret_cast<const int4*>(p.ref)[q] : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int i = 4 * (u * kPlan + threadIdx.x);
      const int v[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int live = i + c < p.n_pages && v[c] > 0;
        all += live;
        before += i < (int)blockIdx.x * kChunk ? live : 0;
        below += i + c < n_live ? live : 0;
      }
    }
  } else {
    const int lc = min(max(n_live, 0), p.n_pages - 1) / kChunk;
    for (int c = threadIdx.x; c < (int)gridDim.x; c += kPlan) {
      const int v = m.chunk[c];
      all += v;
      if (c < (int)blockIdx.x) before += v;
      if (c < lc) below += v;
    }
    for (int i = lc * kChunk + threadIdx.x; i < min(n_live, p.n_pages); i += kPlan)
      below += p.ref[i] > 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  below = __reduce_add_sync(0xffffffffu, below);
  all = __reduce_add_sync(0xffffffffu, all);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_int4(before, below, all, 0);
  __syncthreads();
  before = below = all = 0;
#pragma unroll 8
  for (int w = 0; w < kPlan / 32; ++w) {
    before += sums[w].x;
    below += sums[w].y;
    all += sums[w].z;
  }
  if (all != n_live) {                      // the header does not agree with ref
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      m.head[0] = -1;
      m.head[1] = 0;
    }
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    m.head[0] = n_live;
    m.head[1] = n_live - below;
  }
  constexpr int kLive = kChunk / kPlan;
  const int i0 = blockIdx.x * kChunk + threadIdx.x * kLive;   // consecutive pages of a thread
  int live[kLive], sum = 0;
#pragma unroll
  for (int u = 0; u < kLive; ++u) {
    live[u] = i0 + u < p.n_pages && p.ref[i0 + u] > 0;
    sum += live[u];
  }
  int t;
  int k = before + block_scan<kPlan>(sum, wsum, t);          // pages in use before i
#pragma unroll
  for (int u = 0; u < kLive; ++u) {
    const int i = i0 + u;
    if (i < p.n_pages) {
      if (!live[u] && i < n_live) m.hole[i - k] = i;
      if (live[u] && i >= n_live) {
        m.rank[i] = k - below;
        m.mover[k - below] = i;
      }
    }
    k += live[u];
  }
}

// ------------------------------------------------------------ page copies by the TMA engine
//
// A page's K and V are copied in chunks of CH bytes through a ring of S stages in shared
// memory, by bulk copies that one thread of the CTA issues: loads run S/2 chunks ahead of
// the stores.  2 CTAs an SM, 64 KB each.  Bound by HBM, read + write: a compaction of 2.06 GB
// takes 333 us with its scan and tables (6.2 TB/s).  The copies alone, in a program of their
// own: 318 us (6,480 GB/s; the device's own copy of as much 313 us), loads and stores of 16
// bytes a thread 334 to 359 us over 2 to 8 CTAs of 256 threads an SM and 4 or 8 vectors a
// thread, 32 KB chunks (6 stages, 1 CTA an SM) 319 us, 8 KB ones 344 to 392 us.
constexpr int kMove = 128;        // threads: thread 0 copies, the others do the bookkeeping
constexpr int kMovePerSm = 2;
constexpr int kRing = 65536;

template <int S>
struct Ring {
  uint64_t full[S];
  unsigned char* to[S];
};

// One thread: chunks blockIdx, blockIdx + grid, ... of `n` page copies, so that the chunks
// in flight are neighbours (1,777 scattered pages of 128 KB, the copies alone: 80 us, whole
// pages by a CTA 93 us).  pair(i, from, to) names copy i
// and says whether it is made.
template <int CH, int S, typename Pair>
ETA_DEV void copy_ring(const Pool& p, int n, unsigned char* smem, Ring<S>* ring, Pair pair) {
  constexpr int L = S / 2;        // loads ahead of the stores
  const int half = p.Hkv * p.blk * p.d * 2 / CH;      // chunks of a page of one pool
  for (int s = 0; s < S; ++s) mbar_init(&ring->full[s], 1);
  fence_mbar_init();
  const long long total = 2ll * half * n;
  long long c = blockIdx.x;
  uint32_t loads = 0, stores = 0;
  auto load = [&]() -> bool {     // the next chunk into its stage; false: no more
    for (; c < total; c += gridDim.x) {
      const int i = (int)(c / (2 * half)), u = (int)(c - 2ll * half * i);
      int from = 0, to = 0;
      if (!pair(i, from, to)) continue;
      const int v = u >= half;
      unsigned char* pool = reinterpret_cast<unsigned char*>(v ? p.V : p.K);
      const size_t off = (size_t)(u - v * half) * CH, page = (size_t)half * CH;
      const int s = loads % S;
      ring->to[s] = pool + to * page + off;
      mbar_arrive_expect_tx(&ring->full[s], CH);
      bulk_g2s(smem + s * CH, pool + from * page + off, CH, &ring->full[s]);
      ++loads;
      c += gridDim.x;
      return true;
    }
    return false;
  };
  bool more = true;
  while (more && loads < L) more = load();
  while (stores < loads) {
    const int s = stores % S;
    if (!mbar_wait(&ring->full[s], (stores / S) & 1u, nullptr)) {
      // a lost copy: wait, bounded, for the others in flight and give up
      set_status(p.status, ETA_DEVSTAT_TIMEOUT);
      for (uint32_t k = stores + 1; k < loads; ++k)
        mbar_wait(&ring->full[k % S], (k / S) & 1u, nullptr);
      break;
    }
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(ring->to[s]),
                 "r"(smem_u32(smem + s * CH)), "r"(CH)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    ++stores;
    // the next load's stage was last stored from S - L groups ago
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(S - L) : "memory");
    if (more) more = load();
  }
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <int CH>
__global__ void __launch_bounds__(kMove) compact_move_kernel(const Pool p, const Moves m) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Ring<kRing / CH> ring;
  ETA_PDL_ENTRY();
  const int n_live = m.head[0], moves = m.head[1];
  if (n_live < 0) return;
  if (threadIdx.x == 0) {
    copy_ring<CH, kRing / CH>(p, moves, smem, &ring, [&](int r, int& from, int& to) {
      from = m.mover[r];
      to = m.hole[r];
      return true;
    });
    return;
  }
  if (threadIdx.x < 32) return;
  const long long step = (long long)gridDim.x * (kMove - 32);
  const long long t0 = (long long)blockIdx.x * (kMove - 32) + threadIdx.x - 32;
  for (long long i = t0; i < (long long)p.B * p.NB; i += step) {
    const int page = p.table[i];
    if (page < n_live || page >= p.n_pages) continue;
    const int r = m.rank[page];
    if (r >= 0 && r < moves && m.mover[r] == page) p.table[i] = m.hole[r];
    else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);       // a free page in a table
  }
  for (long long i = t0; i < p.n_pages - n_live; i += step)
    p.free_list[i] = p.n_pages - 1 - (int)i;
  for (long long r = t0; r < moves; r += step) {
    const int from = m.mover[r];
    p.ref[m.hole[r]] = p.ref[from];
    p.ref[from] = 0;
  }
}

// ------------------------------------------------------------------------------- copy
// mark[page]: the first pair that writes it (or n), -1 for the source of a pair.
__global__ void __launch_bounds__(kPlan)
copy_plan_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                 int n, int32_t* mark) {
  ETA_PDL_ENTRY();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (page_ok(p, dst[i])) mark[dst[i]] = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (page_ok(p, dst[i])) atomicMin(&mark[dst[i]], i);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (page_ok(p, src[i])) mark[src[i]] = -1;
}

// OWN: few pairs and bytes of a small pool, every CTA checks them all by itself before it copies,
// with a bit a page in the ring's memory; else mark is copy_plan_kernel's.
template <int CH, bool OWN>
__global__ void __launch_bounds__(kMove)
copy_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            int n, const int32_t* __restrict__ mark) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Ring<kRing / CH> ring;
  __shared__ int2 s_pair[OWN ? kOwnCheck : 1];        // (from, to); from -1: refused
  ETA_PDL_ENTRY();
  if constexpr (OWN) {
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem);
    const int nq = (p.n_pages + 127) / 128;
    for (int i = threadIdx.x; i < nq; i += kMove)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kMove) {
      const int f = src[j], t = dst[j];
      const bool ok = page_ok(p, f) && page_ok(p, t);
      s_pair[j] = make_int2(ok ? f : -1, t);
      if (page_ok(p, f)) atomicOr(&bits[f >> 5], 1u << (f & 31));
    }
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kMove) {    // a dst that is a src
      const int t = s_pair[j].y;
      if (page_ok(p, t) && (bits[t >> 5] >> (t & 31) & 1u)) s_pair[j].x = -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nq; i += kMove)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    bool twice = false;                               // any dst that is named twice
    for (int j = threadIdx.x; j < n; j += kMove) {
      const int t = s_pair[j].y;
      if (page_ok(p, t)) twice |= atomicOr(&bits[t >> 5], 1u << (t & 31)) >> (t & 31) & 1u;
    }
    if (__syncthreads_or(twice)) {                    // rare: the first pair counts
      for (int j = threadIdx.x; j < n; j += kMove) {
        const int t = s_pair[j].y;
        for (int k = 0; k < j; ++k)
          if (s_pair[k].y == t) s_pair[j].x = -1;
      }
      __syncthreads();
    }
    // the copies' writes come after these reads and writes of the ring's memory
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (threadIdx.x != 0) return;
  copy_ring<CH, kRing / CH>(p, n, smem, &ring, [&](int i, int& from, int& to) {
    bool bad;
    if constexpr (OWN) {
      const int2 r = s_pair[i];
      from = r.x;
      to = r.y;
      bad = from < 0;
    } else {
      from = src[i];
      to = dst[i];
      bad = !page_ok(p, from) || !page_ok(p, to) || mark[to] != i;
    }
    if (bad) set_status(p.status, ETA_DEVSTAT_BAD_ROW);
    return !bad;
  });
}

// --------------------------------------------------------------------------- host side
struct WsPages {
  size_t rec, first, done, head, chunk, bitmap, hole, mover, rank, total;
};

inline WsPages ws_pages(const eta_dims_t* d, int32_t n_pages) {
  WsPages w;
  size_t x = 0;
  const size_t np = (size_t)n_pages;
  w.rec = x;    x = align_up(x + ((size_t)d->B + 1) * 8, 256);
  w.first = x;  x = align_up(x + (size_t)d->B * 4, 256);
  w.done = x;   x += 256;
  w.head = x;   x += 256;
  w.chunk = x;  x = align_up(x + (np + kChunk - 1) / kChunk * 4, 256);
  w.bitmap = x; x = align_up(x + (np + 31) / 32 * 4, 256);
  w.hole = x;   x = align_up(x + np * 4, 256);
  w.mover = x;  x = align_up(x + np * 4, 256);
  w.rank = x;   x = align_up(x + np * 4, 256);
  w.total = x;
  return w;
}

inline Pool make_pool(const eta_dims_t* d, int32_t n_pages, int32_t* state, eta_bf16_t* K,
                      eta_bf16_t* V, int32_t* status) {
  const PageLayout L = page_layout(d, n_pages);
  Pool p;
  p.B = d->B; p.NB = num_blocks(d); p.n_pages = n_pages; p.Hkv = d->Hkv; p.blk = d->blk;
  p.d = d->d;
  p.header = state + L.header; p.lengths = state + L.lengths; p.table = state + L.table;
  p.ref = state + L.ref; p.free_list = state + L.free_list;
  p.K = K; p.V = V; p.status = status;
  return p;
}

// Arguments common to the calls that change a cache.
inline eta_status_t check_call(const eta_dims_t* d, int32_t n_pages, const void* state,
                               const void* ws, size_t ws_bytes) {
  const eta_status_t st = check_pool(d, n_pages);
  if (st != ETA_OK) return st;
  if (!state || !aligned16(state)) return ETA_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < ws_pages(d, n_pages).total) return ETA_ERR_WORKSPACE;
  return ETA_OK;
}

template <typename T>
inline T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// Chunks of 16 KB, or of 8 KB where a page of one pool is no multiple of 16 KB.
inline bool wide_chunks(const eta_dims_t* d) { return d->Hkv * d->blk * d->d * 2 % 16384 == 0; }

template <auto Kern, typename... Args>
inline eta_status_t launch_move(dim3 grid, cudaStream_t s, Args... args) {
  if (!set_smem_once<Kern>(kRing)) return ETA_ERR_CUDA;
  return launch_k(Kern, grid, dim3(kMove), kRing, s, args...);
}

inline int copy_grid(int64_t items, int per_sm = 8) {
  const int64_t most = (int64_t)std::max(sm_count(), 1) * per_sm;
  return (int)std::max<int64_t>(1, std::min(items, most));
}

}  // namespace pg
}  // namespace eta

using namespace eta;
using namespace eta::pg;

extern "C" size_t eta_page_state_words(const eta_dims_t* dims, int32_t n_pages) {
  if (check_pool(dims, n_pages) != ETA_OK) return 0;
  return page_layout(dims, n_pages).words;
}

extern "C" size_t eta_page_workspace_size(const eta_dims_t* dims, int32_t n_pages) {
  if (check_pool(dims, n_pages) != ETA_OK) return 0;
  return ws_pages(dims, n_pages).total;
}

extern "C" eta_status_t eta_page_state_offsets(const eta_dims_t* dims, int32_t n_pages,
                                               int64_t* out) {
  const eta_status_t st = check_pool(dims, n_pages);
  if (st != ETA_OK) return st;
  if (!out) return ETA_ERR_INVALID_ARG;
  const PageLayout L = page_layout(dims, n_pages);
  out[0] = (int64_t)L.header; out[1] = (int64_t)L.lengths; out[2] = (int64_t)L.table;
  out[3] = (int64_t)L.ref; out[4] = (int64_t)L.free_list;
  return ETA_OK;
}

extern "C" eta_status_t eta_page_init(const eta_dims_t* dims, int32_t n_pages, int32_t* state,
                                      void* stream) {
  const eta_status_t st = check_pool(dims, n_pages);
  if (st != ETA_OK) return st;
  if (!state || !aligned16(state)) return ETA_ERR_INVALID_ARG;
  const Pool p = make_pool(dims, n_pages, state, nullptr, nullptr, nullptr);
  const int64_t words = std::max<int64_t>((int64_t)p.B * p.NB, n_pages);
  return launch_k(init_kernel, dim3(copy_grid((words + kCopy - 1) / kCopy)), dim3(kCopy), 0,
                  static_cast<cudaStream_t>(stream), p);
}

extern "C" eta_status_t eta_page_append(const eta_dims_t* dims, int32_t n_pages, int32_t* state,
                                        eta_bf16_t* K_pool, eta_bf16_t* V_pool,
                                        const eta_bf16_t* k_new, const eta_bf16_t* v_new,
                                        const int32_t* cu_new, int32_t n_new, void* ws,
                                        size_t ws_bytes, int32_t* dev_status, void* stream) {
  eta_status_t st = check_call(dims, n_pages, state, ws, ws_bytes);
  if (st != ETA_OK) return st;
  if (n_new < 0 || !cu_new || !K_pool || !V_pool) return ETA_ERR_INVALID_ARG;
  if (n_new == 0) return ETA_OK;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) || !aligned16(K_pool) ||
      !aligned16(V_pool))
    return ETA_ERR_INVALID_ARG;
  const Pool p = make_pool(dims, n_pages, state, K_pool, V_pool, dev_status);
  const WsPages w = ws_pages(dims, n_pages);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int2* rec = at<int2>(ws, w.rec);
  int32_t* done = at<int32_t>(ws, w.done);
  const uint4* kn = reinterpret_cast<const uint4*>(k_new);
  const uint4* vn = reinterpret_cast<const uint4*>(v_new);
  const int per = kCopy / 32;
  const dim3 grid(copy_grid(((int64_t)n_new + per - 1) / per, 4));
  if (dims->B <= kLocal)
    return launch_k(append_kernel<true>, grid, dim3(kCopy), 0, s, p, cu_new, (int)n_new,
                    (const int2*)nullptr, done, kn, vn);
  st = launch_k(append_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, cu_new, (int)n_new, rec);
  if (st != ETA_OK) return st;
  return launch_k(append_kernel<false>, grid, dim3(kCopy), 0, s, p, cu_new, (int)n_new,
                  (const int2*)rec, done, kn, vn);
}

extern "C" eta_status_t eta_page_fork(const eta_dims_t* dims, int32_t n_pages, int32_t* state,
                                      eta_bf16_t* K_pool, eta_bf16_t* V_pool, const int32_t* src,
                                      const int32_t* dst, int32_t n, void* ws, size_t ws_bytes,
                                      int32_t* dev_status, void* stream) {
  eta_status_t st = check_call(dims, n_pages, state, ws, ws_bytes);
  if (st != ETA_OK) return st;
  if (n < 0 || n > dims->B) return ETA_ERR_INVALID_ARG;
  if (n == 0) return ETA_OK;
  if (!src || !dst || !K_pool || !V_pool || !aligned16(K_pool) || !aligned16(V_pool))
    return ETA_ERR_INVALID_ARG;
  const Pool p = make_pool(dims, n_pages, state, K_pool, V_pool, dev_status);
  const WsPages w = ws_pages(dims, n_pages);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int2* rec = at<int2>(ws, w.rec);
  int32_t* done = at<int32_t>(ws, w.done);
  const dim3 grid(n, 8);
  if (dims->B <= kLocal && n <= kLocalPairs)
    return launch_k(fork_kernel<true>, grid, dim3(kCopy), 0, s, p, src, dst, (int)n,
                    (const int2*)nullptr, done);
  st = launch_k(fork_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, src, dst, (int)n,
                at<int32_t>(ws, w.first), rec);
  if (st != ETA_OK) return st;
  return launch_k(fork_kernel<false>, grid, dim3(kCopy), 0, s, p, src, dst, (int)n,
                  (const int2*)rec, done);
}

extern "C" eta_status_t eta_page_free(const eta_dims_t* dims, int32_t n_pages, int32_t* state,
                                      const int32_t* rows, int32_t n, void* ws, size_t ws_bytes,
                                      int32_t* dev_status, void* stream) {
  eta_status_t st = check_call(dims, n_pages, state, ws, ws_bytes);
  if (st != ETA_OK) return st;
  if (n < 0 || n > dims->B) return ETA_ERR_INVALID_ARG;
  if (n == 0) return ETA_OK;
  if (!rows) return ETA_ERR_INVALID_ARG;
  const Pool p = make_pool(dims, n_pages, state, nullptr, nullptr, dev_status);
  const WsPages w = ws_pages(dims, n_pages);
  const int parts = std::min((p.NB + kCopy - 1) / kCopy, 8);
  return launch_k(free_kernel, dim3(n, parts), dim3(kCopy), 0, static_cast<cudaStream_t>(stream),
                  p, rows, (int)n, at<uint32_t>(ws, w.bitmap), at<int32_t>(ws, w.done));
}

extern "C" eta_status_t eta_page_compact(const eta_dims_t* dims, int32_t n_pages, int32_t* state,
                                         eta_bf16_t* K_pool, eta_bf16_t* V_pool, void* ws,
                                         size_t ws_bytes, int32_t* dev_status, void* stream) {
  eta_status_t st = check_call(dims, n_pages, state, ws, ws_bytes);
  if (st != ETA_OK) return st;
  if (!K_pool || !V_pool || !aligned16(K_pool) || !aligned16(V_pool)) return ETA_ERR_INVALID_ARG;
  const Pool p = make_pool(dims, n_pages, state, K_pool, V_pool, dev_status);
  const WsPages w = ws_pages(dims, n_pages);
  const Moves m{at<int32_t>(ws, w.head), at<int32_t>(ws, w.chunk), at<int32_t>(ws, w.hole),
                at<int32_t>(ws, w.mover), at<int32_t>(ws, w.rank)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int nc = (n_pages + kChunk - 1) / kChunk;
  if (nc > kOwnCount &&
      (st = launch_k(compact_count_kernel, dim3(nc), dim3(kPlan), 0, s, p, m)) != ETA_OK)
    return st;
  st = nc > kOwnCount
           ? launch_k(compact_plan_kernel<false>, dim3(nc), dim3(kPlan), 0, s, p, m)
           : launch_k(compact_plan_kernel<true>, dim3(nc), dim3(kPlan), 0, s, p, m);
  if (st != ETA_OK) return st;
  const dim3 grid(copy_grid(n_pages, kMovePerSm));
  return wide_chunks(dims) ? launch_move<compact_move_kernel<16384>>(grid, s, p, m)
                           : launch_move<compact_move_kernel<8192>>(grid, s, p, m);
}

extern "C" eta_status_t eta_page_copy(const eta_dims_t* dims, int32_t n_pages, eta_bf16_t* K_pool,
                                      eta_bf16_t* V_pool, const int32_t* src, const int32_t* dst,
                                      int32_t n, void* ws, size_t ws_bytes, int32_t* dev_status,
                                      void* stream) {
  eta_status_t st = check_pool(dims, n_pages);
  if (st != ETA_OK) return st;
  const WsPages w = ws_pages(dims, n_pages);
  if (!ws || !aligned16(ws) || ws_bytes < w.total) return ETA_ERR_WORKSPACE;
  if (n < 0) return ETA_ERR_INVALID_ARG;
  if (n == 0) return ETA_OK;
  if (!src || !dst || !K_pool || !V_pool || !aligned16(K_pool) || !aligned16(V_pool))
    return ETA_ERR_INVALID_ARG;
  const Pool p = [&] {
    Pool x = {};
    x.n_pages = n_pages; x.Hkv = dims->Hkv; x.blk = dims->blk; x.d = dims->d;
    x.K = K_pool; x.V = V_pool; x.status = dev_status;
    return x;
  }();
  int32_t* mark = at<int32_t>(ws, w.rank);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = wide_chunks(dims);
  const int64_t bytes = (int64_t)n * 2 * dims->Hkv * dims->blk * dims->d * 2;
  const dim3 grid(copy_grid(bytes / 8192, kMovePerSm));
  const int32_t* no_mark = nullptr;
  if (n <= kOwnCheck && bytes <= kOwnBytes && n_pages <= kRing * 8)
    return wide ? launch_move<copy_kernel<16384, true>>(grid, s, p, src, dst, (int)n, no_mark)
                : launch_move<copy_kernel<8192, true>>(grid, s, p, src, dst, (int)n, no_mark);
  if ((st = launch_k(copy_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, src, dst, (int)n, mark)) !=
      ETA_OK)
    return st;
  const int32_t* marks = mark;
  return wide ? launch_move<copy_kernel<16384, false>>(grid, s, p, src, dst, (int)n, marks)
              : launch_move<copy_kernel<8192, false>>(grid, s, p, src, dst, (int)n, marks);
}
