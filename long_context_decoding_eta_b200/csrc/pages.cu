// Bookkeeping and data movement of a paged KV cache: append, fork, free, compact, copy
// (include/eta.h, "Paged caches").  No counterpart in the ETA pages.
//
// Every call is two or three launches: a plan that decides everything from the state
// before the call (one CTA where the decision is a scan over rows or pairs), then
// kernels that carry it out in parallel.  Page numbers come from prefix sums and
// bitmaps, never from the arrival order of atomics, so the same calls always give the
// same tables; the only atomics are integer counts whose order does not matter.
// The data kernels move whole 16-byte vectors; they are bound by HBM (read + write of
// the moved tokens), the bookkeeping by launch latency.
#include <algorithm>

#include "eta_common.cuh"
#include "paged_host.h"

namespace eta {
namespace pg {

constexpr int kPlan = 1024;       // threads of a one-CTA plan
constexpr int kCopy = 256;        // threads of a data-moving CTA
constexpr int kChunk = 4096;      // pages per CTA of the compaction's scan

struct Pool {
  int B, NB, n_pages, Hkv, blk, d;
  int32_t *header, *lengths, *table, *ref, *free_list;
  eta_bf16_t *K, *V;
  int32_t* status;
};

// Exclusive prefix sum of v over the kPlan threads of the CTA; total is the sum.
ETA_DEV int block_scan(int v, int* wsum, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = wsum[lane];
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += y;
    }
    wsum[lane] = wi - w;
    if (lane == 31) wsum[32] = wi;
  }
  __syncthreads();
  const int r = wsum[warp] + incl - v;
  total = wsum[32];
  __syncthreads();
  return r;
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
// Per row: the length before the call (-1: refused, or nothing to do) and how many pages
// the rows before it take; rec[B] holds the free count before the call, and whether the
// offsets were refused.
__global__ void __launch_bounds__(kPlan)
append_plan_kernel(const Pool p, const int32_t* __restrict__ cu, int n_new, int2* rec) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[33];
  __shared__ int s_used;
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  if (threadIdx.x == 0) s_used = 0;
  bool bad = false;                          // offsets out of order: nothing is appended
  for (int b = threadIdx.x; b < p.B; b += kPlan)
    bad |= cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > n_new;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) set_status(p.status, ETA_DEVSTAT_BAD_LENGTH);
  int carry = 0;
  for (int base = 0; base < p.B; base += kPlan) {
    const int b = base + threadIdx.x;
    int need = 0, len = 0, n = 0;
    bool ok = false;
    if (b < p.B && !bad) {
      const int c0 = cu[b], c1 = cu[b + 1];
      len = p.lengths[b];
      if (len < 0 || len > p.NB * p.blk || c1 - c0 > p.NB * p.blk - len) {
        set_status(p.status, ETA_DEVSTAT_BAD_LENGTH);
      } else {
        n = c1 - c0;
        ok = n > 0;
        if (ok && len % p.blk != 0) {
          const int last = p.table[(size_t)b * p.NB + len / p.blk];
          if (!page_ok(p, last) || p.ref[last] != 1) {
            set_status(p.status, ETA_DEVSTAT_BAD_ROW);
            ok = false;
          }
        }
        if (ok) need = blocks_of(len + n, p.blk) - blocks_of(len, p.blk);
      }
    }
    int total;
    const int before = carry + block_scan(need, wsum, total);
    if (need > 0) {
      if (before + need <= n_free) {
        atomicMax(&s_used, before + need);
      } else {
        set_status(p.status, ETA_DEVSTAT_NO_PAGE);
        ok = false;
      }
    }
    if (b < p.B) {
      rec[b] = make_int2(ok ? len : -1, before);
      if (ok) p.lengths[b] = len + n;
    }
    carry += total;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    rec[p.B] = make_int2(n_free, bad);
    p.header[0] = n_free - s_used;
  }
}

// One warp per new token: finds its row, its page (from the table, or from the free
// list where the block is new), and writes the token's Hkv key and value vectors.  The
// warp of a new block's first token enters the page into the table.
__global__ void __launch_bounds__(kCopy)
append_kernel(const Pool p, const int32_t* __restrict__ cu, int n_new,
              const int2* __restrict__ rec, const uint4* __restrict__ kn,
              const uint4* __restrict__ vn) {
  ETA_PDL_ENTRY();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5);
  if (t >= n_new) return;
  if (rec[p.B].y) return;                    // nothing is appended
  int lo = 0, hi = p.B - 1;                  // the last row with cu[row] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int b = lo, c0 = cu[b];
  const int2 r = rec[b];
  if (t < c0 || t >= cu[b + 1] || r.x < 0) return;
  const int pos = r.x + t - c0;
  const int j = pos / p.blk, slot = pos - j * p.blk;
  if (!ETA_IN_BOUNDS(j, p.NB, p.status)) return;
  const int first_new = blocks_of(r.x, p.blk);
  int page;
  if (j >= first_new) {
    const int k = rec[p.B].x - 1 - (r.y + j - first_new);
    if (!ETA_IN_BOUNDS(k, p.n_pages, p.status)) return;
    page = p.free_list[k];
    if (page_ok(p, page) && lane == 0 && (slot == 0)) {
      p.table[(size_t)b * p.NB + j] = page;
      p.ref[page] = 1;
    }
  } else {
    page = p.table[(size_t)b * p.NB + j];
  }
  if (!page_ok(p, page)) {
    if (lane == 0) set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
    return;
  }
  const int vd = p.d / 8, nv = p.Hkv * vd;   // 16-byte vectors of a token's keys
  for (int i = lane; i < nv; i += 32) {
    const int g = i / vd, x = i - g * vd;
    const size_t to = (((size_t)page * p.Hkv + g) * p.blk + slot) * vd + x;
    const uint4 a = kn[(size_t)t * nv + i], c = vn[(size_t)t * nv + i];
    reinterpret_cast<uint4*>(p.K)[to] = a;
    reinterpret_cast<uint4*>(p.V)[to] = c;
  }
}

// ------------------------------------------------------------------------------- fork
// rec[i]: the source's length (-1: the pair is refused) and the new last page (-1: none).
__global__ void __launch_bounds__(kPlan)
fork_plan_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                 int n, int32_t* first, int2* rec) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[33];
  __shared__ int s_used;
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  if (threadIdx.x == 0) s_used = 0;
  // the first pair that names each dst
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int t = dst[i];
    if (t >= 0 && t < p.B) first[t] = 0x7fffffff;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int t = dst[i];
    if (t >= 0 && t < p.B) atomicMin(&first[t], i);
  }
  __syncthreads();
  int carry = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int need = 0, len = -1;
    if (i < n) {
      const int f = src[i], t = dst[i];
      if (f >= 0 && f < p.B && t >= 0 && t < p.B && __ldcg(first + t) == i &&
          p.lengths[t] == 0) {
        len = min(max(p.lengths[f], 0), p.NB * p.blk);
        need = len % p.blk != 0;
      } else {
        set_status(p.status, ETA_DEVSTAT_BAD_ROW);
      }
    }
    int total;
    const int before = carry + block_scan(need, wsum, total);
    int page = -1;
    if (need) {
      if (before < n_free) {
        page = p.free_list[n_free - 1 - before];
        atomicMax(&s_used, before + 1);
      } else {
        set_status(p.status, ETA_DEVSTAT_NO_PAGE);
        len = -1;
      }
    }
    if (i < n) rec[i] = make_int2(len, page);
    carry += total;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.header[0] = n_free - s_used;
}

// Grid (pairs, parts): the parts of a pair share its table row and its last page.
__global__ void __launch_bounds__(kCopy)
fork_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            const int2* __restrict__ rec) {
  ETA_PDL_ENTRY();
  const int i = blockIdx.x;
  const int2 r = rec[i];
  if (r.x < 0) return;
  const int f = src[i], t = dst[i];
  const int full = r.x / p.blk, part = r.x - full * p.blk;
  const int tid = blockIdx.y * kCopy + threadIdx.x, step = gridDim.y * kCopy;
  for (int j = tid; j < full; j += step) {
    const int page = p.table[(size_t)f * p.NB + j];
    p.table[(size_t)t * p.NB + j] = page;
    if (page_ok(p, page)) atomicAdd(&p.ref[page], 1);
    else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
  }
  if (tid == 0) {
    p.lengths[t] = r.x;
    if (part && page_ok(p, r.y)) {
      p.table[(size_t)t * p.NB + full] = r.y;
      p.ref[r.y] = 1;
    }
  }
  if (part) {
    const int old = p.table[(size_t)f * p.NB + full];
    if (!page_ok(p, old) || !page_ok(p, r.y)) {
      if (tid == 0) set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      return;
    }
    const int vd = p.d / 8, per = part * vd;       // 16-byte vectors of one head's tokens
    for (int x = tid; x < p.Hkv * per; x += step) {
      const int g = x / per, y = x - g * per;
      const size_t from = ((size_t)old * p.Hkv + g) * p.blk * vd + y;
      const size_t to = ((size_t)r.y * p.Hkv + g) * p.blk * vd + y;
      const uint4 a = reinterpret_cast<const uint4*>(p.K)[from];
      const uint4 c = reinterpret_cast<const uint4*>(p.V)[from];
      reinterpret_cast<uint4*>(p.K)[to] = a;
      reinterpret_cast<uint4*>(p.V)[to] = c;
    }
  }
}

// ------------------------------------------------------------------------------- free
// Grid (rows, parts).  A table entry is taken with an exchange, so a row named twice
// gives its pages back once; a page whose last reference goes is marked in the bitmap.
__global__ void __launch_bounds__(kCopy)
free_kernel(const Pool p, const int32_t* __restrict__ rows, uint32_t* bitmap) {
  ETA_PDL_ENTRY();
  const int b = rows[blockIdx.x];
  if (b < 0 || b >= p.B) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_status(p.status, ETA_DEVSTAT_BAD_ROW);
    return;
  }
  const int nb = min(blocks_of(max(p.lengths[b], 0), p.blk), p.NB);
  for (int j = blockIdx.y * kCopy + threadIdx.x; j < nb; j += gridDim.y * kCopy) {
    const int page = atomicExch(&p.table[(size_t)b * p.NB + j], -1);
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

// One CTA: pushes the marked pages in descending order, clears the bitmap, and empties
// the rows.
__global__ void __launch_bounds__(kPlan)
free_push_kernel(const Pool p, const int32_t* __restrict__ rows, int n, uint32_t* bitmap) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[33];
  const int n_free = min(max(p.header[0], 0), p.n_pages);
  const int nw = (p.n_pages + 31) / 32;
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int b = rows[i];
    if (b >= 0 && b < p.B) p.lengths[b] = 0;
  }
  int at = n_free;
  for (int base = 0; base < nw; base += kPlan) {
    const int w = nw - 1 - (base + (int)threadIdx.x);
    uint32_t m = w >= 0 ? bitmap[w] : 0u;
    int total;
    int k = at + block_scan(__popc(m), wsum, total);
    if (m) bitmap[w] = 0u;
    while (m) {
      const int bit = 31 - __clz(m);
      m &= ~(1u << bit);
      if (k < p.n_pages) p.free_list[k] = w * 32 + bit;
      else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      ++k;
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

ETA_DEV int chunk_live(const Pool& p, int c, int end, int* wsum) {
  int v = 0;
  for (int i = c * kChunk + threadIdx.x; i < min(end, p.n_pages); i += kPlan) v += p.ref[i] > 0;
  int total;
  block_scan(v, wsum, total);
  return total;
}

__global__ void __launch_bounds__(kPlan) compact_count_kernel(const Pool p, const Moves m) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[33];
  const int live = chunk_live(p, blockIdx.x, (blockIdx.x + 1) * kChunk, wsum);
  if (threadIdx.x == 0) m.chunk[blockIdx.x] = live;
}

__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Pool p, const Moves m) {
  ETA_PDL_ENTRY();
  __shared__ int wsum[33];
  const int nc = gridDim.x;
  int before = 0, below = 0, all = 0;       // live before this chunk, before n_live's, in all
  const int n_live = p.n_pages - p.header[0];
  const int lc = min(max(n_live, 0), p.n_pages - 1) / kChunk;
  for (int c = threadIdx.x; c < nc; c += kPlan) {
    const int v = m.chunk[c];
    all += v;
    if (c < (int)blockIdx.x) before += v;
    if (c < lc) below += v;
  }
  int t;
  block_scan(before, wsum, t);
  before = t;
  block_scan(below, wsum, t);
  below = t;
  block_scan(all, wsum, t);
  all = t;
  if (all != n_live) {                      // the header does not agree with ref
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
      m.head[0] = -1;
      m.head[1] = 0;
    }
    return;
  }
  below += chunk_live(p, lc, n_live, wsum);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    m.head[0] = n_live;
    m.head[1] = n_live - below;
  }
  for (int base = 0; base < kChunk; base += kPlan) {
    const int i = blockIdx.x * kChunk + base + threadIdx.x;
    const int live = i < p.n_pages && p.ref[i] > 0;
    const int k = before + block_scan(live, wsum, t);     // pages in use before i
    if (i < p.n_pages) {
      if (!live && i < n_live) m.hole[i - k] = i;
      if (live && i >= n_live) {
        m.rank[i] = k - below;
        m.mover[k - below] = i;
      }
    }
    before += t;
  }
}

// Copies `vecs` 16-byte vectors with the CTA's threads, four loads in flight each.
ETA_DEV void copy_vecs(uint4* __restrict__ to, const uint4* __restrict__ from, int vecs) {
  int i = threadIdx.x;
  for (; i + 3 * kCopy < vecs; i += 4 * kCopy) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = from[i + u * kCopy];
#pragma unroll
    for (int u = 0; u < 4; ++u) to[i + u * kCopy] = v[u];
  }
  for (; i < vecs; i += kCopy) to[i] = from[i];
}

ETA_DEV void copy_page(const Pool& p, int to, int from) {
  const int vecs = p.Hkv * p.blk * p.d / 8;
  copy_vecs(reinterpret_cast<uint4*>(p.K) + (size_t)to * vecs,
            reinterpret_cast<const uint4*>(p.K) + (size_t)from * vecs, vecs);
  copy_vecs(reinterpret_cast<uint4*>(p.V) + (size_t)to * vecs,
            reinterpret_cast<const uint4*>(p.V) + (size_t)from * vecs, vecs);
}

__global__ void __launch_bounds__(kCopy) compact_move_kernel(const Pool p, const Moves m) {
  ETA_PDL_ENTRY();
  const int n_live = m.head[0], moves = m.head[1];
  if (n_live < 0) return;
  const long long step = (long long)gridDim.x * kCopy;
  const long long t0 = (long long)blockIdx.x * kCopy + threadIdx.x;
  for (long long i = t0; i < (long long)p.B * p.NB; i += step) {
    const int page = p.table[i];
    if (page < n_live || page >= p.n_pages) continue;
    const int r = m.rank[page];
    if (r >= 0 && r < moves && m.mover[r] == page) p.table[i] = m.hole[r];
    else set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);       // a free page in a table
  }
  for (long long i = t0; i < p.n_pages - n_live; i += step)
    p.free_list[i] = p.n_pages - 1 - (int)i;
  for (int r = blockIdx.x; r < moves; r += gridDim.x) {
    const int from = m.mover[r], to = m.hole[r];
    copy_page(p, to, from);
    if (threadIdx.x == 0) {
      p.ref[to] = p.ref[from];
      p.ref[from] = 0;
    }
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

__global__ void __launch_bounds__(kCopy)
copy_kernel(const Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
            int n, const int32_t* __restrict__ mark) {
  ETA_PDL_ENTRY();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int f = src[i], t = dst[i];
    if (!page_ok(p, f) || !page_ok(p, t) || mark[t] != i) {
      if (threadIdx.x == 0) set_status(p.status, ETA_DEVSTAT_BAD_ROW);
      continue;
    }
    copy_page(p, t, f);
  }
}

// --------------------------------------------------------------------------- host side
struct WsPages {
  size_t rec, first, head, chunk, bitmap, hole, mover, rank, total;
};

inline WsPages ws_pages(const eta_dims_t* d, int32_t n_pages) {
  WsPages w;
  size_t x = 0;
  const size_t np = (size_t)n_pages;
  w.rec = x;    x = align_up(x + ((size_t)d->B + 1) * 8, 256);
  w.first = x;  x = align_up(x + (size_t)d->B * 4, 256);
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

inline int copy_grid(int64_t items) {
  const int64_t most = (int64_t)std::max(sm_count(), 1) * 8;   // 8 CTAs of 256 threads an SM
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
  st = launch_k(append_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, cu_new, (int)n_new, rec);
  if (st != ETA_OK) return st;
  const int per = kCopy / 32;
  return launch_k(append_kernel, dim3((n_new + per - 1) / per), dim3(kCopy), 0, s, p, cu_new,
                  (int)n_new, (const int2*)rec, reinterpret_cast<const uint4*>(k_new),
                  reinterpret_cast<const uint4*>(v_new));
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
  st = launch_k(fork_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, src, dst, (int)n,
                at<int32_t>(ws, w.first), rec);
  if (st != ETA_OK) return st;
  return launch_k(fork_kernel, dim3(n, 8), dim3(kCopy), 0, s, p, src, dst, (const int2*)rec);
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
  uint32_t* bitmap = at<uint32_t>(ws, ws_pages(dims, n_pages).bitmap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int parts = std::min((p.NB + kCopy - 1) / kCopy, 8);
  st = launch_k(free_kernel, dim3(n, parts), dim3(kCopy), 0, s, p, rows, bitmap);
  if (st != ETA_OK) return st;
  return launch_k(free_push_kernel, dim3(1), dim3(kPlan), 0, s, p, rows, (int)n, bitmap);
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
  if ((st = launch_k(compact_count_kernel, dim3(nc), dim3(kPlan), 0, s, p, m)) != ETA_OK) return st;
  if ((st = launch_k(compact_plan_kernel, dim3(nc), dim3(kPlan), 0, s, p, m)) != ETA_OK) return st;
  return launch_k(compact_move_kernel, dim3(copy_grid(n_pages)), dim3(kCopy), 0, s, p, m);
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
  if ((st = launch_k(copy_plan_kernel, dim3(1), dim3(kPlan), 0, s, p, src, dst, (int)n, mark)) !=
      ETA_OK)
    return st;
  return launch_k(copy_kernel, dim3(copy_grid(n)), dim3(kCopy), 0, s, p, src, dst, (int)n,
                  (const int32_t*)mark);
}
