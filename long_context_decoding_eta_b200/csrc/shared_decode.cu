// Decode attention for a batch whose rows share long prefixes, each prefix read once for
// all of its rows (include/eta.h, eta_shared_decode).  The gate is Eq. 2-3 of the
// evolve.pub review of arXiv 2609.20888 (Methodology Assessment), on every key.
//
// A softmax over disjoint key sets joins exactly: with per-set maxima m_i, sums l_i =
// sum e^(s - m_i) and weighted sums o_i, M = max m_i gives o = sum e^(m_i - M) o_i /
// sum e^(m_i - M) l_i.  So the queries of all rows of a group (rows x G heads of one KV
// head) attend over the prefix together, as the M side of tensor-core tiles, every row
// attends over its own remaining keys, and the parts are joined at the end.  The prefix
// then costs its bytes once, and rows * G flops per byte: HBM-bound for small groups,
// bound by the tensor cores and the exponentials from about 256 (row, head) pairs on.
//
// Three launches:
//   shared_plan_kernel   (one CTA) the work list.  An item is (group, KV head, up to 256
//                        (row, head) pairs) over the prefix, or (row, KV head) over the
//                        row's own keys, in key tiles of 128.  The items' costs, laid end
//                        to end, are cut into equal shares, one per SM.
//   shared_attend_kernel one CTA per share: 384 threads, warps 0-3 / 4-7 the softmax of
//                        streams A / B, warp 8 the TMA producer, warps 9 / 10 their Q K^T,
//                        warp 11 the P V of both.
//                        S_x = Q K^T and O_x += P V with M = 128 queries, 64 keys at a
//                        time: one half of a key tile is in the softmax while the other's
//                        products run.  A thread owns a query row, so no row statistic is
//                        exchanged.
//                        Two streams keep the tensor cores busy while the other stream's
//                        exponentials run: with more than 128 pairs A and B are two query
//                        tiles that share every K/V tile; else they take alternate K/V
//                        tiles of the one query tile, with accumulators of their own.
//                        P overwrites S in tensor memory.
//   shared_combine_kernel  joins the parts of every (row, head).
//
// 64 rows of 16 / 4 heads of 128 over a 128K-token prefix and up to 1,024 own tokens each,
// bf16 output: 114 us a call with new inputs (103 as a replayed graph, part of the keys in
// L2) for a floor of 52 (341 MB); the attend kernel alone runs at 45% of HBM, 47% of the
// tensor pipe and 46% of the SFU, bound by the chain Q K^T - softmax - P V of its streams.
// 4 rows of 2,048 + 64 tokens: 23 us, three launches' latency.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>

#include "combine_dev.cuh"
#include "decode_tc.cuh"
#include "eta_common.cuh"
#include "paged_host.h"
#include "tma_host.h"

namespace eta {
namespace sd {

using tc::fence_async_smem;
using tc::smem_desc;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_2d;

constexpr int TILE = 128;                       // query rows and keys of a tile
constexpr int SUB = 64;                         // keys of a TMA box (half a tile)
constexpr int HALF = TILE * 128;                // [128 rows x 64 dims] bf16 = 16 KB
constexpr int NSEG = 4;                         // segment records in flight
constexpr int NT = 384;
constexpr int kPlan = 1024;
constexpr int kTmemCols = 512;
constexpr uint32_t kIssueLimit = 1u << 26;      // polls for a load to be issued
constexpr float kRescale = 8.0f;                // rescale O when the max grows by > 8 (e^8)
constexpr float kLog2e = 1.4426950408889634f;
enum Gate { NONE = 0, HARD = 1, SOFT = 2 };

// ------------------------------------------------------------------------- work list
// Costs in about half microseconds, as measured (64 rows over 128K tokens, 4 KV heads): a key
// tile of up to 256 or 128 queries, a key tile of a row's own, and what a row's own item
// costs besides (its few tiles cannot fill the pipeline).  An item's tiles begin at 0 and
// seg + t * cost; a CTA has the tiles that begin in its share of the costs.  With few
// tiles every tile costs 1, so that they spread over all CTAs: 4 rows of 2,048 + 64 tokens
// are 80 tiles for 80 CTAs, where the costs above left 44 of them three each.
// The same costs serve every form; of {pair, single, own, seg} = {4, 3, 3, 4}, {4, 2, 2, 4},
// {4, 4, 4, 4} and {1, 1, 1, 0} they are best or close to it, but for soft gates (us, 64 rows of
// 16 / 4 heads of 128: one group of 128K tokens, bf16, no gate 103, 112, 107, 103; 32 groups of
// one page and 4,096 own tokens, fp32, no gate 129, 134, 128, 128; four groups of up to 32K
// tokens, bf16, no gate 90, 90, 104, 103; the same in fp32 with a soft gate 215, 180, 266, 253).
struct Costs {
  int pair, single, own, seg;
  ETA_DEV int own_begin(int t) const { return t ? seg + t * own : 0; }
  ETA_DEV int own_cost(int nt) const { return nt ? seg + nt * own : 0; }
  // the smallest share: every share inside an item has a tile's begin
  ETA_DEV int gap() const { return max(max(pair, single), own + seg); }
};
ETA_DEV Costs costs_of(int tiles, int P) {
  return tiles <= 2 * P ? Costs{1, 1, 1, 0} : Costs{4, 3, 3, 4};
}

struct GroupRec {
  int off;        // its first item's place in the costs
  int nt;         // key tiles of an item; 0: nothing is shared
  int cost;       // of a key tile
  int npairs;     // 256-row items per KV head
  int row0, nrows;
  int leader;     // the row whose table names the prefix pages
  int nb;         // shared blocks
  int rows;       // partial rows of a slot
  int base;       // first partial row of the group's slots
  int cf;         // CTA of its first tile
};

struct RowRec {
  int off;        // its first item's place, counted behind all prefixes
  int nt;         // key tiles per KV head
  int start;      // first block that the row reads by itself
  int group;      // the group it shares a prefix with, or -1
};

struct Head {
  int share, suffix_base;
  Costs cost;
};

// What a CTA begins with: its share [a, e) of the costs, the group (or n_groups + row) at
// a, and the cost of all prefixes.
struct CtaRec {
  int a, e, item, prefix_cost;
};

struct Ws {
  Head* head;
  GroupRec* grp;
  RowRec* row;
  CtaRec* cta;
  float* part_ml;
  float* part_o;
};

struct PlanParams {
  int B, Hkv, G, NB, blk, n_groups, n_pages, P;
  const int32_t *lengths, *group_off, *prefix_len, *table;
  Ws ws;
  int32_t* status;
};

ETA_DEV int2 add2(int2 a, int2 b) { return make_int2(a.x + b.x, a.y + b.y); }

ETA_DEV int2 cta_scan(int2 v, int2* wsum, int2& total) {   // exclusive, over kPlan threads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto incl_scan = [&](int2 x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int2 y = make_int2(__shfl_up_sync(0xffffffffu, x.x, o),
                               __shfl_up_sync(0xffffffffu, x.y, o));
      if (lane >= o) x = add2(x, y);
    }
    return x;
  };
  const int2 incl = incl_scan(v);
  __syncthreads();                              // wsum's last readers are done
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  const int2 w = incl_scan(wsum[lane]);         // every warp alike
  total = make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
  const int2 before = make_int2(__shfl_sync(0xffffffffu, w.x, (warp + 31) & 31),
                                __shfl_sync(0xffffffffu, w.y, (warp + 31) & 31));
  return make_int2((warp ? before.x : 0) + incl.x - v.x, (warp ? before.y : 0) + incl.y - v.y);
}

__global__ void __launch_bounds__(kPlan) shared_plan_kernel(const PlanParams p) {
  ETA_PDL_ENTRY();
  __shared__ int2 wsum[32];
  __shared__ int s_tiles;                       // of all items
  if (threadIdx.x == 0) s_tiles = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cap = p.NB * p.blk;
  bool bad = false;
  for (int g = threadIdx.x; g < p.n_groups; g += kPlan) {
    const int r0 = p.group_off[g], r1 = p.group_off[g + 1];
    bad |= r0 < 0 || r1 < r0 || r1 > p.B;
  }
  for (int b = threadIdx.x; b < p.B; b += kPlan) {
    p.ws.row[b].start = 0;
    p.ws.row[b].group = -1;
    const int len = p.lengths[b];
    if (len < 0 || len > cap) set_status(p.status, ETA_DEVSTAT_BAD_LENGTH);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 &&
      (bad || p.group_off[0] != 0 || p.group_off[p.n_groups] != p.B))
    set_status(p.status, ETA_DEVSTAT_BAD_ROW);
  // a warp per group: who shares, and whose table is read
  for (int g = warp; g < p.n_groups; g += kPlan / 32) {
    const int r0 = bad ? 0 : p.group_off[g], r1 = bad ? 0 : p.group_off[g + 1];
    int pre = p.prefix_len[g];
    if (pre < 0 || pre > cap) {
      if (lane == 0) set_status(p.status, ETA_DEVSTAT_BAD_LENGTH);
      pre = min(max(pre, 0), cap);
    }
    const int nb = pre / p.blk;
    int first = 0x7fffffff, count = 0;
    if (nb > 0)
      for (int r = r0 + lane; r < r1; r += 32)
        if (min(p.lengths[r], cap) >= nb * p.blk) {
          first = min(first, r);
          ++count;
        }
    first = __reduce_min_sync(0xffffffffu, first);
    count = __reduce_add_sync(0xffffffffu, count);
    const bool share = count > 1;
    if (share)
      for (int r = r0 + lane; r < r1; r += 32)
        if (min(p.lengths[r], cap) >= nb * p.blk) {
          p.ws.row[r].start = nb;
          p.ws.row[r].group = g;
        }
    if constexpr (kChecked)                      // the rows hold the pages that are read
      if (share)
        for (int r = first; r < r1; ++r) {
          if (min(p.lengths[r], cap) < nb * p.blk) continue;
          bool other = false;
          for (int j = lane; j < nb; j += 32) {
            const int page = p.table[(size_t)first * p.NB + j];   // out of range: BAD_BLOCK
            other |= (unsigned)page < (unsigned)p.n_pages &&
                     page != p.table[(size_t)r * p.NB + j];
          }
          if (other) set_status(p.status, ETA_DEVSTAT_BAD_ROW);
        }
    if (lane == 0) {
      GroupRec rec;
      int tiles;
      const int rows = (r1 - r0) * p.G;
      rec.nt = share ? (nb * p.blk + TILE - 1) / TILE : 0;
      rec.cost = rows > TILE;                    // pair or single: see below
      tiles = p.Hkv * rec.nt * ((rows + 2 * TILE - 1) / (2 * TILE));
      rec.npairs = (rows + 2 * TILE - 1) / (2 * TILE);
      rec.row0 = r0;
      rec.nrows = r1 - r0;
      rec.leader = first;
      rec.nb = nb;
      rec.rows = rec.npairs > 1 ? 2 * TILE : rows <= TILE ? 2 * rows : rows;
      rec.off = rec.base = rec.cf = 0;
      p.ws.grp[g] = rec;
      if (tiles) atomicAdd(&s_tiles, tiles);
    }
  }
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += kPlan) {
    const int b = b0 + threadIdx.x;
    int nt = 0;
    if (b < p.B) {
      const int len = min(max(p.lengths[b], 0), cap);
      nt = (max(len - p.ws.row[b].start * p.blk, 0) + TILE - 1) / TILE;
      p.ws.row[b].nt = nt;
    }
    nt = __reduce_add_sync(0xffffffffu, nt);
    if (lane == 0 && nt) atomicAdd(&s_tiles, nt * p.Hkv);
  }
  __syncthreads();
  const Costs w = costs_of(s_tiles, p.P);
  // places in the costs: of the groups (x) and of the rows (y, counted from zero)
  int2 carry = make_int2(0, 0), total;
  for (int i0 = 0; i0 < max(p.n_groups, p.B); i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int2 n = make_int2(0, 0);
    if (i < p.n_groups) {
      GroupRec g = p.ws.grp[i];
      g.cost = g.cost ? w.pair : w.single;
      p.ws.grp[i].cost = g.cost;
      n.x = p.Hkv * g.npairs * g.nt * g.cost;
    }
    if (i < p.B) n.y = p.Hkv * w.own_cost(p.ws.row[i].nt);
    const int2 off = add2(carry, cta_scan(n, wsum, total));
    if (i < p.n_groups) p.ws.grp[i].off = off.x;
    if (i < p.B) p.ws.row[i].off = off.y;
    carry = add2(carry, total);
  }
  const int prefix_cost = carry.x, costs = carry.x + carry.y;
  const int share = max((costs + p.P - 1) / p.P, w.gap());
  for (int c = threadIdx.x; c < p.P; c += kPlan) {
    p.ws.cta[c].a = min(c * share, costs);
    p.ws.cta[c].e = min(c * share + share, costs);
    p.ws.cta[c].prefix_cost = prefix_cost;
  }
  // where a group's partial results go
  carry = make_int2(0, 0);
  for (int g0 = 0; g0 < p.n_groups; g0 += kPlan) {
    const int g = g0 + threadIdx.x;
    int2 rows = make_int2(0, 0);
    int cf = 0;
    if (g < p.n_groups) {
      const int off = p.ws.grp[g].off, items = p.Hkv * p.ws.grp[g].npairs;
      const int n = items * p.ws.grp[g].nt * p.ws.grp[g].cost;
      if (n > 0) {
        cf = off / share;
        rows.x = ((off + n - 1) / share - cf + items) * p.ws.grp[g].rows;
      }
    }
    const int2 base = add2(carry, cta_scan(rows, wsum, total));
    if (g < p.n_groups) {
      p.ws.grp[g].base = base.x;
      p.ws.grp[g].cf = cf;
    }
    carry = add2(carry, total);
  }
  // the item that every CTA starts in: of a group by a warp, of a row by a thread
  for (int g = warp; g < p.n_groups; g += kPlan / 32) {
    const GroupRec r = p.ws.grp[g];
    const int off = r.off, n = p.Hkv * r.npairs * r.nt * r.cost;
    for (int c = (off + share - 1) / share + lane; c * share < off + n; c += 32)
      p.ws.cta[c].item = g;
  }
  for (int b = threadIdx.x; b < p.B; b += kPlan) {
    const int off = prefix_cost + p.ws.row[b].off, n = p.Hkv * w.own_cost(p.ws.row[b].nt);
    for (int c = (off + share - 1) / share; c * share < off + n; ++c)
      p.ws.cta[c].item = p.n_groups + b;
  }
  if (threadIdx.x == 0) *p.ws.head = Head{share, carry.x, w};
}

// ---------------------------------------------------------------------------- attend
struct Seg {
  int live;             // 0: no more segments
  int pair;             // streams are two query tiles (else alternate key tiles of one)
  int ntiles, base;     // key tiles, and the CTA's running number of the first
  int row0;             // batch row of query row 0 of stream A
  int kvh;
  int mA, mB;           // valid query rows of the streams' tiles
  int partA, partB;     // first partial row of each stream
  int check;            // prefix: rows that do not share it are left out
  int flip;             // single: the stream of the first key tile
};

// What the MMA warps need of a key tile, a word per tile in a ring: written before the
// tile's K is counted in `issued`.
enum TileFlags {
  kPairTile = 1,        // both streams take it; else stream T & 1
  kFirst = 2,           // the first of its segment for every stream that takes it
  kQSlot = 4,           // single: the query slot is 1
  kQRel1 = 8,           // arrivals at the query slot's `empty` behind this tile's Q K^T: one,
  kQRel2 = 16,          // or two
  kQPhase0 = 32, kQPhase1 = 64,   // the phase of each query slot's load
};
constexpr int NTILE = 16;                       // tile words in flight (at most 7 are)

// Jobs (key tiles) of stream x in a segment, and the tile of job j.
ETA_DEV int jobs_of(const Seg& s, int x) {
  return s.pair ? s.ntiles : (s.ntiles + 1 - (x ^ s.flip)) >> 1;
}
ETA_DEV int tile_of(const Seg& s, int x, int j) { return s.pair ? j : 2 * j + (x ^ s.flip); }

template <int D>
struct Misc {
  static constexpr int NSLOT = D == 128 ? 5 : 10;
  uint64_t q_full[2], q_empty[2], kv_full[NSLOT], kv_empty[NSLOT];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_free[2];   // [stream][half tile]
  uint64_t seg_full[NSEG], seg_empty[NSEG], fin[3];
  Seg seg[NSEG];
  int2 nv[NSLOT];       // of a V slot: valid keys of the tile's two 64-key halves
  int tile[NTILE];      // TileFlags
  int issued;           // loads of K and V tiles under way so far
  int end;              // key tiles of the CTA, once known
  uint32_t tmem_base;
  int abort_flag;
};

// Shared memory: two query tiles, then a ring of slots of one K or V tile each; tile T of
// the CTA has its K in slot 2 T and its V in slot 2 T + 1, modulo the slots.  K and V are
// apart because K is done with long before V: its slot loads again while the softmax runs.
template <int D>
struct Cfg {
  static constexpr int NH = D / 64;                     // 64-dim boxes
  static constexpr int SLOT = NH * HALF;                // one query, key or value tile
  static constexpr int NSLOT = Misc<D>::NSLOT;
  static constexpr int OFF_Q = 0;                       // tiles A, B
  static constexpr int OFF_KV = 2 * SLOT;
  static constexpr int OFF_MISC = OFF_KV + NSLOT * SLOT;
  static constexpr int SMEM = OFF_MISC + (int)sizeof(Misc<D>) + 1024;
  ETA_DEV static int kslot(int t) { return 2 * t % NSLOT; }
  ETA_DEV static int kload(int t) { return 2 * t / NSLOT; }
  ETA_DEV static int vslot(int t) { return (2 * t + 1) % NSLOT; }
  ETA_DEV static int vload(int t) { return (2 * t + 1) / NSLOT; }
};
static_assert(Cfg<128>::SMEM <= 227 * 1024, "shared decode shared memory");

struct AttendParams {
  int B, Hq, Hkv, G, NB, blk, n_pages, n_groups;
  float scale, invT;
  const float* tau;
  const int32_t *table, *lengths;
  Ws ws;
  int part_rows;        // partial rows of the workspace (the checked build's limit)
  int32_t* status;
};

// kind::f16, D fp32, A/B bf16, M = 128
template <int N>
constexpr uint32_t idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// The MMA warps run with all their lanes, so that descriptors are computed in uniform
// registers, and one elected lane issues: 8 MMAs take 229 cycles to issue this way, 546 from
// a branch of one lane.
ETA_DEV uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(e));
  return e;
}
ETA_DEV void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id,
                    uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead)
      : "memory");
}
ETA_DEV void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id,
                    uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(id), "r"(acc), "r"(lead)
      : "memory");
}
ETA_DEV void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          smem_u32(bar)),
      "r"(lead)
      : "memory");
}

ETA_DEV void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

ETA_DEV void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::
          "r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

ETA_DEV void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}

// Waits for the thread's loads; the 32 values are operands so that their use stays behind.
ETA_DEV void tmem_wait_ld32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])::"memory");
}

ETA_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

ETA_DEV float ex2_approx(float x) {             // 2^x on the SFU; -inf gives 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
ETA_DEV float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
ETA_DEV float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Box of 64 dims x G heads x `rows` batch rows of q [B, Hq, d]: the query rows packed as
// (row, head), 128 bytes each.
ETA_DEV void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Whether phase `parity` of `bar` is over, without waiting.
ETA_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A whole warp's wait: one try (which itself waits a while), then the bounded polls.  As one
// loop 108 us where the two take 105 (64 rows over 128K tokens, bf16, no gate); with the polls
// out of line 107, but 170 for 175 with the soft gate and 99 for 101 at d = 64.
ETA_DEV bool warp_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
ETA_DEV bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         warp_wait_slow(bar, parity, abort);
}

// Waits until load `item` (tile T's K is 2 T, its V 2 T + 1) has been issued; false too
// when the CTA has no such tile.  A whole warp's wait.
ETA_DEV bool wait_issued_slow(volatile int* issued, volatile int* end, int item,
                              volatile int* abort) {
  uint32_t polls = 0;
  bool ok = true;
  while (ok && *issued <= item)
    ok = !(*end <= item / 2 || ++polls > kIssueLimit || *abort);
  return __all_sync(0xffffffffu, ok);
}
ETA_DEV bool wait_issued(volatile int* issued, volatile int* end, int item,
                         volatile int* abort) {
  const bool ok = __all_sync(0xffffffffu, *issued > item) ||
                  wait_issued_slow(issued, end, item, abort);
  __threadfence_block();
  return ok;
}

// The gate on 32 scores of a query row, in raw units (see the softmax).
struct GateArgs {
  float tau_raw, tau, scale, f;
  float zero;           // 0, or NaN where tau is
};
template <int GATE>
ETA_DEV void gate32(float* v, const GateArgs& g) {
  if constexpr (GATE == HARD) {
    // a selection: a flag times the score would make NaN of an infinite score
#pragma unroll
    for (int u = 0; u < 32; ++u) v[u] = v[u] >= g.tau_raw ? v[u] : 0.f;
  } else if constexpr (GATE == SOFT) {
    // s / (1 + e), e = 2^x: two keys share a reciprocal, 1 / b0 = b1 / (b0 b1).  x is at most
    // 63, which keeps b0 b1 finite (s * 2^-63 stands for 0); the minimum also keeps a NaN (a
    // key past the end) away from its neighbour.  s * 0 makes NaN of an infinite score, which
    // the quotient would.
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      const float2 s2 = make_float2(v[u], v[u + 1]);
      const float2 x = __fmul2_rn(
          __ffma2_rn(s2, make_float2(g.scale, g.scale), make_float2(-g.tau, -g.tau)),
          make_float2(g.f, g.f));
      const float2 b = __fadd2_rn(make_float2(ex2_approx(fminf(x.x, 63.f)),
                                              ex2_approx(fminf(x.y, 63.f))),
                                  make_float2(1.f, 1.f));
      const float r = rcp_approx(b.x * b.y);
      const float2 w = __fmul2_rn(make_float2(b.y, b.x), make_float2(r, r));
      const float2 y = __ffma2_rn(s2, w, __fmul2_rn(s2, make_float2(g.zero, g.zero)));
      v[u] = y.x;
      v[u + 1] = y.y;
    }
  }
}

// Running maxima of 32 scores, in four independent chains.
ETA_DEV void max32(const float* v, float* pm) {
#pragma unroll
  for (int u = 0; u < 32; u += 2) pm[(u >> 1) & 3] = fmax3(pm[(u >> 1) & 3], v[u], v[u + 1]);
}

// 32 weights e^(scale * (u - m)) = 2^(u * c1 + nm), summed into l2 and rounded to NS
// bf16 terms (each the rounding of what those before it leave), two keys a register.
template <int NS>
ETA_DEV void exp32(const float* v, float c1, float nm, float2& l2, uint32_t (&w)[NS][16]) {
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const float2 a = __ffma2_rn(make_float2(v[2 * u], v[2 * u + 1]), make_float2(c1, c1),
                                make_float2(nm, nm));
    float2 r = make_float2(ex2_approx(a.x), ex2_approx(a.y));
    l2 = __fadd2_rn(l2, r);
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(r.x, r.y);
      w[k][u] = *reinterpret_cast<const uint32_t*>(&t);
      const float2 f = __bfloat1622float2(t);
      r.x -= f.x;
      r.y -= f.y;
    }
  }
}

// Tensor-memory columns: stream x's scores of half h at x * S_STREAM + h * S_HALF, P over
// them in NS terms of 32 columns; O behind.  Three terms take 96 columns: at d = 128, where
// O needs half of tensor memory, the two halves of a stream then share theirs and take
// turns.
template <int D, int NS>
struct Tm {
  static constexpr int S_STREAM = D == 64 ? 192 : 128;
  static constexpr int S_HALF = D == 64 ? 96 : NS == 1 ? 64 : 0;
  static constexpr int O = 2 * S_STREAM, O_STREAM = D;
  static_assert(O + 2 * O_STREAM <= kTmemCols, "tensor memory");
  static_assert(NS * 32 <= (S_HALF ? S_HALF : S_STREAM), "P terms");
};

// GATE: Gate.  NS: the bf16 terms of P, each half a step of 8 bits behind the one before.  One
// (2^-8) for a bf16 output, whose own rounding is as coarse: the largest error is then 1.4 times
// that of fp32 weights (2.3e-3 and 1.65e-3, 64 rows over 128K tokens).  Three (2^-24) for an
// fp32 one, where two (2^-16) left an error of 2e-6, eight times the plain fp32 form's.
template <int D, int GATE, int NS>
__global__ void __launch_bounds__(NT, 1)
shared_attend_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmQ1,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttendParams p) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Misc<D>* ms = reinterpret_cast<Misc<D>*>(smem + C::OFF_MISC);
  volatile int* abort_flag = &ms->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(&ms->kv_full[s], 1);
      mbar_init(&ms->kv_empty[s], 2);           // both streams, or one of them twice
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&ms->q_full[x], 1);
      mbar_init(&ms->q_empty[x], 2);
      mbar_init(&ms->fin[x], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&ms->s_full[x][h], 1);
        mbar_init(&ms->p_full[x][h], 4);
        mbar_init(&ms->pv_done[x][h], 1);
      }
      mbar_init(&ms->o_free[x], 4);
    }
    for (int s = 0; s < NSEG; ++s) {
      mbar_init(&ms->seg_full[s], 1);
      mbar_init(&ms->seg_empty[s], 8);          // the softmax warps
    }
    mbar_init(&ms->fin[2], 1);
    ms->issued = 0;
    ms->end = 0x7fffffff;
    ms->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&ms->tmem_base)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  using M = Tm<D, NS>;
  ETA_PDL_ENTRY();

  if (warp == 8) {
    // ------------------------------------------------------------------ TMA producer
    // The whole warp: 32 pages are looked up at a time, a tile's boxes are issued by a
    // lane each.  Every variable but the lane's own page and box is the same in all lanes.
    const CtaRec me = p.ws.cta[blockIdx.x];
    const Head hd = *p.ws.head;
    const int suffix_base = hd.suffix_base;
    const Costs w = hd.cost;
    const int e = me.e, shift = p.blk == 64 ? 6 : 7;
    int pos = me.a, at = me.item;
    bool ok = true;
    int nseg = 0, slots = 0;                     // segments begun, K/V slots loaded so far
    int qn[2] = {0, 0};                          // loads of each query slot so far
    // The lane's 64-key piece of a row: piece k0 / 64 + lane; its page, or -2 past the end.
    auto page_of = [&](int row, int k0, int end) -> int {
      const int key = k0 + lane * SUB;
      return key < end ? p.table[(size_t)row * p.NB + (key >> shift)] : -2;
    };
    auto clamped = [&](int len) { return min(max(len, 0), p.NB << shift); };
    // The row being read by itself and the one after it: record, length and first pages,
    // asked for a row ahead (a row can be one tile for each KV head).
    RowRec r = {}, nr = {};
    int len = 0, nlen = 0, pg_row = -2, npg_row = -2, b = -1;
    bool npg = false;
    auto next_row = [&] {
      if (b + 1 < p.B) {
        nr = p.ws.row[b + 1];
        nlen = p.lengths[b + 1];
      }
    };
    auto next_pages = [&] {
      if (!npg && b + 1 < p.B) npg_row = page_of(b + 1, nr.start << shift, clamped(nlen));
      npg = true;
    };
    // every lane polls; all agree on the outcome
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return warp_wait(bar, parity, abort_flag);
    };
    while (ok) {
      Seg s = {};
      int key0 = 0, key_end = 0, trow = 0, mrows = 0, pg = -2;
      while (pos < e && pos < me.prefix_cost) {
        const GroupRec g = p.ws.grp[at];
        const int items = p.Hkv * g.npairs, ic = g.nt * g.cost, local = pos - g.off;
        if (ic == 0 || local >= items * ic) {
          if (++at >= p.n_groups) {              // only when the next place is a row's
            pos = me.prefix_cost;
            break;
          }
          continue;
        }
        // the first tile that begins at pos or behind it
        const int item = local / ic, t = (local - item * ic + g.cost - 1) / g.cost;
        pos = g.off + item * ic + t * g.cost;
        if (t == g.nt || pos >= e) continue;
        const int pair = item % g.npairs, i0 = pair * 2 * TILE;
        const int left = g.nrows * p.G - i0;
        s.live = 1;
        s.pair = left > TILE;
        s.ntiles = min(g.nt - t, (e - pos + g.cost - 1) / g.cost);
        s.row0 = g.row0 + i0 / p.G;
        s.kvh = item / g.npairs;
        s.mA = min(left, TILE);
        s.mB = s.pair ? min(left - TILE, TILE) : s.mA;
        s.partA = g.base + ((int)blockIdx.x - g.cf + item) * g.rows;
        s.partB = s.partA + (!s.pair && g.npairs == 1 ? s.mA : TILE);
        s.check = 1;
        key0 = t * TILE;
        key_end = g.nb << shift;
        trow = g.leader;
        mrows = TILE;
        pg = page_of(trow, key0, key_end);
        pos += s.ntiles * g.cost;
        break;
      }
      while (!s.live && pos < e) {
        if (b < 0) {
          b = max(at - p.n_groups, 0);
          r = p.ws.row[b];
          len = clamped(p.lengths[b]);
          next_row();
          pg_row = page_of(b, r.start << shift, len);
        }
        int local = pos - me.prefix_cost - r.off;
        if (local >= w.own_cost(r.nt) * p.Hkv) {
          if (b + 1 >= p.B) {                    // cannot happen: a place has an item
            pos = e;
            break;
          }
          next_pages();
          ++b;
          r = nr;
          len = clamped(nlen);
          pg_row = npg_row;
          npg = false;
          next_row();
          continue;
        }
        const int ic = w.own_cost(r.nt), g = local / ic, base = pos - local + g * ic;
        local -= g * ic;
        // the first tile that begins at pos or behind it, and the first behind the share
        const int t = local == 0 ? 0 : max((local - w.seg + w.own - 1) / w.own, 1);
        const int te = min(max((e - base - w.seg + w.own - 1) / w.own, 1), r.nt);
        pos = base + (t >= r.nt ? ic : w.own_begin(t));
        if (t >= r.nt || pos >= e) continue;
        s.live = 1;
        s.pair = 0;
        s.ntiles = te - t;
        s.row0 = b;
        s.kvh = g;
        s.mA = s.mB = p.G;
        s.partA = suffix_base + ((int)blockIdx.x + b * p.Hkv + g) * 2 * p.G;
        s.partB = s.partA + p.G;
        key0 = (r.start << shift) + t * TILE;
        key_end = len;
        trow = b;
        mrows = p.G;
        pg = t == 0 ? pg_row : page_of(b, key0, len);
        pos = base + (te == r.nt ? ic : w.own_begin(te));
      }
      s.base = slots / 2;
      // Tile T of single segments is stream T & 1's, so that a stream's next tile is never
      // more than two on: its K is then loaded into a slot that an earlier tile frees.
      s.flip = s.base & 1;
      const int qslot = nseg & 1;
      const int qflags = (s.pair ? kPairTile : qslot * kQSlot) | (qn[0] & 1) * kQPhase0 |
                         (qn[1] & 1) * kQPhase1;
      // the record, then the first key tile, the queries, and the other tiles
      const int sl = nseg % NSEG;
      if (!wwait(&ms->seg_empty[sl], ((uint32_t)(nseg / NSEG) & 1u) ^ 1u)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        ms->seg[sl] = s;
        mbar_arrive(&ms->seg_full[sl]);
      }
      if (!s.live) {
        if (lane == 0) *(volatile int*)&ms->end = s.base;
        break;
      }
      __syncwarp();
      int npages = -2;                           // the lane's page of the next 16 tiles
      const int u = lane & 1, hb = (lane >> 1) * 64;   // the lane's box: key half, dims
      for (int t = 0; t < s.ntiles && ok; ++t) {
        const int k0 = key0 + t * TILE, i = t & 15;
        if (i == 0) {
          if (t > 0) pg = npages;
          npages = page_of(trow, k0 + 16 * TILE, key_end);
        }
        const int pg0 = __shfl_sync(0xffffffffu, pg, 2 * i);
        const int pg1 = __shfl_sync(0xffffffffu, pg, 2 * i + 1);
        int nv0 = max(min(key_end - k0, SUB), 0), nv1 = max(min(key_end - k0 - SUB, SUB), 0);
        if ((nv0 > 0 && (unsigned)pg0 >= (unsigned)p.n_pages) ||
            (nv1 > 0 && (unsigned)pg1 >= (unsigned)p.n_pages)) {
          if (lane == 0) set_status(p.status, ETA_DEVSTAT_BAD_BLOCK);
          if ((unsigned)pg0 >= (unsigned)p.n_pages) nv0 = 0;
          if ((unsigned)pg1 >= (unsigned)p.n_pages) nv1 = 0;
        }
        const uint32_t bytes = (uint32_t)(((nv0 > 0) + (nv1 > 0)) * C::NH * (HALF / 2));
        const bool mine = lane < 2 * C::NH && (u ? nv1 : nv0) > 0;
        const int key = k0 + u * SUB;
        const int y = (((u ? pg1 : pg0) * p.Hkv + s.kvh) << shift) + (key & (p.blk - 1));
#pragma unroll
        for (int v = 0; v < 2; ++v) {            // K, then V
          const int st = slots % C::NSLOT;
          if (!wwait(&ms->kv_empty[st], ((uint32_t)(slots / C::NSLOT) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (v) {
              ms->nv[st] = make_int2(nv0, nv1);
            } else {
              // both arrivals at a query slot come from the one stream that uses it, or
              // one from each, behind its last tile
              const int last = s.ntiles - 1 - t;
              ms->tile[(slots / 2) % NTILE] =
                  qflags | (t < (s.pair ? 1 : 2) ? kFirst : 0) |
                  (s.pair || s.ntiles == 1 ? (last == 0 ? kQRel2 : 0) : (last < 2 ? kQRel1 : 0));
            }
            mbar_arrive_expect_tx(&ms->kv_full[st], bytes);
            __threadfence_block();
            *(volatile int*)&ms->issued = slots + 1;
          }
          __syncwarp();
          unsigned char* to = smem + C::OFF_KV + st * C::SLOT + (lane >> 1) * HALF + u * (HALF / 2);
          if (mine) {
            if (v) tma_load_2d(to, &tmV, hb, y, &ms->kv_full[st]);
            else tma_load_2d(to, &tmK, hb, y, &ms->kv_full[st]);
          }
          ++slots;
          if (t == 0 && v == 0) {
            // query slots: a pair fills both, a single segment the one of its number
            for (int x = 0; x < 2; ++x) {
              if (!s.pair && x != qslot) continue;
              if (!wwait(&ms->q_empty[x], ((uint32_t)qn[x] & 1u) ^ 1u)) {
                ok = false;
                break;
              }
              if (lane == 0)
                mbar_arrive_expect_tx(&ms->q_full[x], (uint32_t)(mrows * 128 * C::NH));
              __syncwarp();
              ++qn[x];
              const int row = s.row0 + (s.pair && x ? TILE / p.G : 0);
              if (lane < C::NH) {
                unsigned char* q = smem + C::OFF_Q + x * C::SLOT + lane * HALF;
                if (s.check) tma_load_3d(q, &tmQ, lane * 64, s.kvh * p.G, row, &ms->q_full[x]);
                else tma_load_3d(q, &tmQ1, lane * 64, s.kvh * p.G, row, &ms->q_full[x]);
              }
            }
            if (!ok) break;
          }
        }
      }
      ++nseg;
      if (b >= 0) next_pages();                  // the next row's record is here by now
    }
    if (!ok) {
      // wait (bounded) for every copy this warp issued before the CTA exits
      if (lane == 0) set_status(p.status, ETA_DEVSTAT_TIMEOUT);
      *abort_flag = 1;
      for (int k = max(0, slots - C::NSLOT); k < slots; ++k)
        mbar_wait(&ms->kv_full[k % C::NSLOT], (uint32_t)(k / C::NSLOT) & 1u, nullptr);
      for (int x = 0; x < 2; ++x)
        if (qn[x] > 0) mbar_wait(&ms->q_full[x], (uint32_t)(qn[x] - 1) & 1u, nullptr);
    }
    __syncwarp();
  } else if (warp > 8) {
    // ------------------------------------------------------------------ MMA issuers
    // A warp for each stream's Q K^T, which is issued once the stream's S columns (P of the
    // tile before) are free, and one for the P V of both streams, whichever has its P
    // written.  (13 warps leave 128 registers a thread, and the softmax spilled: 161 us for
    // 104 with one warp a stream for both products, 64 rows of 128K tokens.)
    {
      const uint32_t lead = elect_one();
      bool ok = true;                            // the same in all lanes, as all else
      const uint64_t dq = smem_desc(smem_u32(smem + C::OFF_Q), 16, 1024, tc::kSwizzle128);
      const uint64_t dk = smem_desc(smem_u32(smem + C::OFF_KV), 16, 1024, tc::kSwizzle128);
      const uint64_t dv = smem_desc(smem_u32(smem + C::OFF_KV), HALF, 1024, tc::kSwizzle128);
      constexpr uint32_t id = idesc<D>() | (1u << 16);           // V is MN-major
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return warp_wait(bar, parity, abort_flag);
      };
      auto is_issued = [&](int item) -> bool {
        return wait_issued(&ms->issued, &ms->end, item, abort_flag);
      };
      // The flags of tile T.  A barrier's parity also looks over while the phase before is
      // open, and a stream does not follow the loads of the other's tiles: that a load has
      // been issued says that those before it into the same slot are over.  The queries'
      // load is issued between the first tile's K and V.
      auto flags = [&](int T) -> int {
        return __shfl_sync(0xffffffffu, *(volatile int*)&ms->tile[T % NTILE], 0);
      };
      // Q and K of a tile are in
      auto ready = [&](int x, int T, int f) -> bool {
        if (f & kFirst) {
          const int qs = (f & kPairTile) ? x : (f & kQSlot) ? 1 : 0;
          ok = is_issued(2 * T + 1) &&
               wait(&ms->q_full[qs], (f & (qs ? kQPhase1 : kQPhase0)) ? 1u : 0u);
        }
        return ok = ok && wait(&ms->kv_full[C::kslot(T)], (uint32_t)C::kload(T) & 1u);
      };
      // S_h = Q K_h^T of tile T, the stream's n-th
      auto issue_qk = [&](int x, int T, int f, int n, int h) {
        // S_h's columns hold P of the tile before until P V has read it; or of the half before
        if (M::S_HALF == 0 && h == 1) {
          if (ok) ok = wait(&ms->pv_done[x][0], (uint32_t)n & 1u);
        } else if (ok && n > 0) {
          ok = wait(&ms->pv_done[x][M::S_HALF == 0 ? 1 : h], (uint32_t)(n - 1) & 1u);
        }
        if (!ok) return;
        tc_fence_after();
        const int ks = C::kslot(T), qs = (f & kPairTile) ? x : (f & kQSlot) ? 1 : 0;
        const uint64_t dqs = dq + (uint64_t)(qs * (C::SLOT >> 4));
        const uint64_t dks = dk + (uint64_t)(ks * (C::SLOT >> 4) + h * (HALF / 2 >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * HALF + (kk & 3) * 32) >> 4);
          mma_ss(lead, tmem + x * M::S_STREAM + h * M::S_HALF, dqs + off, dks + off,
                 idesc<SUB>(), kk > 0);
        }
        commit(lead, &ms->s_full[x][h]);
        if (h) {
          // a tile's slot is free after two arrivals: a pair's streams each give one
          commit(lead, &ms->kv_empty[ks]);
          if (!(f & kPairTile)) commit(lead, &ms->kv_empty[ks]);
          if (f & (kQRel1 | kQRel2)) commit(lead, &ms->q_empty[qs]);
          if (f & kQRel2) commit(lead, &ms->q_empty[qs]);
        }
      };
      // O += P_h V_h of tile T of stream x (V is in: the softmax waited for it)
      auto issue_pv = [&](int x, int T, int f, int h) {
        const int vs = C::vslot(T);
        if (!(ok = wait(&ms->kv_full[vs], (uint32_t)C::vload(T) & 1u))) return;
        tc_fence_after();
        const uint64_t dvs = dv + (uint64_t)(vs * (C::SLOT >> 4) + h * (HALF / 2 >> 4));
        const uint32_t acc = h == 0 && (f & kFirst) ? 0u : 1u;
#pragma unroll
        for (int term = 0; term < NS; ++term)
#pragma unroll
          for (int kk = 0; kk < SUB / 16; ++kk)
            mma_ts(lead, tmem + M::O + x * M::O_STREAM,
                   tmem + x * M::S_STREAM + h * M::S_HALF + term * 32 + kk * 8,
                   dvs + (uint64_t)(kk * 2048 >> 4), id, (term > 0 || kk > 0) ? 1u : acc);
        commit(lead, &ms->pv_done[x][h]);
        if (h) {
          commit(lead, &ms->kv_empty[vs]);
          if (!(f & kPairTile)) commit(lead, &ms->kv_empty[vs]);
        }
      };
      if (warp < 11) {
        const int x = warp - 9;
        for (int T = 0, n = 0; ok; ++T) {
          if (!is_issued(2 * T)) {
            ok = __all_sync(0xffffffffu, *(volatile int*)&ms->end <= T);
            break;
          }
          const int f = flags(T);
          if (!(f & kPairTile) && (T & 1) != x) continue;
          if (!ready(x, T, f)) break;
          issue_qk(x, T, f, n, 0);
          issue_qk(x, T, f, n, 1);
          ++n;
        }
      } else {
        // per stream: its tile (have), the tile's half, tiles so far, segments begun
        int T[2] = {0, 0}, f[2] = {0, 0}, h[2] = {0, 0}, n[2] = {0, 0}, segs[2] = {0, 0};
        bool have[2] = {false, false}, over[2] = {false, false};
        auto seen = [&](uint64_t* bar, uint32_t parity) -> bool {
          return __all_sync(0xffffffffu, mbar_test(bar, parity));
        };
        uint32_t idle = 0;
        while (ok && !(over[0] && over[1])) {
          bool did = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (over[x] || !ok) continue;
            if (!have[x]) {
              if (!__all_sync(0xffffffffu, *(volatile int*)&ms->issued > 2 * T[x])) {
                over[x] = __all_sync(0xffffffffu, *(volatile int*)&ms->end <= T[x]);
                continue;
              }
              __threadfence_block();
              f[x] = flags(T[x]);
              did = true;
              if (!(f[x] & kPairTile) && (T[x] & 1) != x) {
                ++T[x];
                continue;
              }
              have[x] = true;
            }
            // the stream's last segment has to be read out of O before O begins anew
            if (h[x] == 0 && (f[x] & kFirst) && segs[x] > 0 &&
                !seen(&ms->o_free[x], (uint32_t)(segs[x] - 1) & 1u))
              continue;
            if (!seen(&ms->p_full[x][h[x]], (uint32_t)n[x] & 1u)) continue;
            did = true;
            if (h[x] == 0 && (f[x] & kFirst)) ++segs[x];
            issue_pv(x, T[x], f[x], h[x]);
            if ((h[x] ^= 1) == 0) {
              have[x] = false;
              ++T[x];
              ++n[x];
            }
          }
          idle = did ? 0 : idle + 1;
          if (idle > kIssueLimit || *abort_flag) ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        if (lead) set_status(p.status, ETA_DEVSTAT_TIMEOUT);
        *abort_flag = 1;
      }
      // every MMA issued so far has completed before TMEM is released
      commit(lead, &ms->fin[warp - 9]);
      mbar_wait(&ms->fin[warp - 9], 0, nullptr);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int x = warp >> 2;                     // stream
    const int i = threadIdx.x & (TILE - 1);      // query row of its tile = TMEM lane
    const uint32_t lsel = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tSx = tmem + x * M::S_STREAM + lsel;
    const uint32_t tOx = tmem + M::O + x * M::O_STREAM + lsel;
    const float c1 = p.scale * kLog2e;
    const float resc_raw = kRescale / p.scale;
    bool ok = true;
    int nseg = 0, cnt = 0;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return warp_wait(bar, parity, abort_flag);
    };
    for (;; ++nseg) {
      const int sl = nseg % NSEG;
      if (!wwait(&ms->seg_full[sl], (uint32_t)(nseg / NSEG) & 1u)) { ok = false; break; }
      const Seg s = ms->seg[sl];
      if (!s.live) break;
      const int mine = x == 0 ? s.mA : s.mB;
      const bool active = (warp & 3) * 32 < mine;      // the warp has a valid row
      const int b = s.row0 + (i + (s.pair && x ? TILE : 0)) / p.G, h = s.kvh * p.G + i % p.G;
      const bool valid = i < mine && ETA_IN_BOUNDS(b, p.B, p.status) &&
                         ETA_IN_BOUNDS(h, p.Hq, p.status);
      const bool store = valid && (!s.check || p.ws.row[b].start > 0);   // the row shares
      // Gated logits in raw units u (the gated logit is scale * u), so that the scale
      // folds into the constants: the hard gate keeps s iff s >= tau / scale, the soft
      // gate is s / (1 + 2^((scale * s - tau) * f)), f = -log2(e) / T (the difference first:
      // over a T near zero both terms are infinite), and e^(scale * (u - m)) is
      // 2^(u * c1 - m * c1), c1 = scale * log2(e).  (s / 2 + s / 2 * tanh((s - tau) / 2T)
      // with the approximate tanh takes one transcendental less, but it is off by up to
      // 2^-12 |s|, in lse too, and that grows with the scores.  64 rows over 128K tokens,
      // bf16: 153 us with it, 174 as it is, 189 with a reciprocal for every key.)
      GateArgs ga = {};
      if constexpr (GATE != NONE) {
        const float tau = valid ? p.tau[(size_t)b * p.Hq + h] : 0.f;
        ga.tau_raw = tau / p.scale;
        ga.tau = tau;
        ga.scale = p.scale;
        ga.f = -kLog2e * p.invT;
        ga.zero = isnan(tau) ? tau : 0.f;
      }
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      const int jobs = jobs_of(s, x);
      for (int j = 0; j < jobs; ++j, ++cnt) {
        const int T = s.base + tile_of(s, x, j);
        // V's slot is not loaded again before this tile's P V
        if (!wwait(&ms->s_full[x][0], (uint32_t)cnt & 1u) ||
            !wait_issued(&ms->issued, &ms->end, 2 * T + 1, abort_flag) ||
            !wwait(&ms->kv_full[C::vslot(T)], (uint32_t)C::vload(T) & 1u)) {
          ok = false;
          break;
        }
        const int2 nv = ms->nv[C::vslot(T)];
        if (nv.x < SUB || nv.y < SUB) {          // V rows past the end must be finite
          if ((i & (SUB - 1)) >= (i < SUB ? nv.x : nv.y)) {
            unsigned char* vt = smem + C::OFF_KV + C::vslot(T) * C::SLOT + i * 128;
#pragma unroll
            for (int hh = 0; hh < C::NH; ++hh)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(vt + hh * HALF + c * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();                          // the loads of S are the whole warp's
        }
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (hf && !wwait(&ms->s_full[x][1], (uint32_t)cnt & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (active) {
            const uint32_t tSh = tSx + hf * M::S_HALF;
            const int lim = hf ? nv.y : nv.x;
            float sv[SUB];
            tmem_ld32(tSh, sv);
            tmem_ld32(tSh + 32, sv + 32);
            tmem_wait_ld32(sv);
            tmem_wait_ld32(sv + 32);
            gate32<GATE>(sv, ga);
            gate32<GATE>(sv + 32, ga);
            if (lim < SUB) {                     // keys past the end
#pragma unroll
              for (int c = 0; c < SUB; ++c)
                if (c >= lim) sv[c] = -INFINITY;
            }
            float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            max32(sv, pm);
            max32(sv + 32, pm);
            const float mx = fmaxf(fmax3(pm[0], pm[1], pm[2]), pm[3]);
            // the first keys set the maximum; later ones rescale O (in TMEM) only when it
            // grew by more than kRescale
            float alpha = 1.f;
            bool resc = false;
            if (m == -INFINITY) {
              m = mx;
            } else if (mx > m + resc_raw) {
              alpha = ex2_approx((m - mx) * c1);
              m = mx;
              resc = true;
            }
            if (__any_sync(0xffffffffu, resc && valid)) {
              // P V of the half tile before has to be complete
              if (!wwait(&ms->pv_done[x][hf ^ 1], (uint32_t)(hf ? cnt : cnt - 1) & 1u)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                float ov[32];
                tmem_ld32(tOx + c * 32, ov);
                tmem_wait_ld32(ov);
#pragma unroll
                for (int u = 0; u < 32; ++u) ov[u] *= alpha;
                tmem_st32(tOx + c * 32, reinterpret_cast<const uint32_t*>(ov));
              }
              l2.x *= alpha;
              l2.y *= alpha;
            }
            const float nm = m == -INFINITY ? 0.f : -m * c1;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[NS][16];
              exp32<NS>(sv + 32 * c, c1, nm, l2, w);
#pragma unroll
              for (int k = 0; k < NS; ++k) tmem_st16(tSh + 32 * k + 16 * c, w[k]);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->p_full[x][hf]);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // the segment's partial result of this stream
      if (jobs > 0) {
        if (!wwait(&ms->pv_done[x][1], (uint32_t)(cnt - 1) & 1u)) { ok = false; break; }
        tc_fence_after();
      }
      if (active) {
        // O by 4 dims, the stream's `mine` rows side by side for each: a warp's stores
        // coalesce (a row's own 512 bytes by each thread took 8,000 cycles a segment)
        const int first = x ? s.partB : s.partA;
        const bool in = ETA_RANGE_IN_BOUNDS(first, first + mine, p.part_rows, p.status);
        if (jobs > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float ov[32];
            __syncwarp();                        // together again behind the stores
            tmem_ld32(tOx + c * 32, ov);
            tmem_wait_ld32(ov);
            if (store && in) {
              float4* to = reinterpret_cast<float4*>(p.ws.part_o) + (size_t)first * (D / 4) +
                           c * 8 * mine + i;
#pragma unroll
              for (int u = 0; u < 8; ++u)
                to[u * mine] = make_float4(ov[4 * u], ov[4 * u + 1], ov[4 * u + 2], ov[4 * u + 3]);
            }
          }
        }
        if (store && in)
          reinterpret_cast<float2*>(p.ws.part_ml)[first + i] =
              make_float2(m * p.scale, l2.x + l2.y);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (jobs > 0) mbar_arrive(&ms->o_free[x]);
        mbar_arrive(&ms->seg_empty[sl]);
      }
    }
    if (!ok) {
      if (lane == 0) set_status(p.status, ETA_DEVSTAT_TIMEOUT);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

// --------------------------------------------------------------------------- combine
constexpr int kCombine = 512;
constexpr int kMaxSlots = 1024;

ETA_DEV void store4(float* o, float4 v) { *reinterpret_cast<float4*>(o) = v; }
ETA_DEV void store4(__nv_bfloat16* o, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// One CTA per (row, KV head), its G heads together (their partial rows lie side by side).
// The slots are the CTAs that had a piece of the row's prefix item (one or two streams
// each) and of its own item.  Thread = (slot group, 4 dims, head).
template <int D, int G, typename OutT>
__global__ void __launch_bounds__(kCombine)
shared_combine_kernel(const AttendParams p, OutT* __restrict__ o, float* __restrict__ lse) {
  ETA_PDL_ENTRY();
  constexpr int VEC = G * D / 4, NG = kCombine / VEC, NW = kCombine / 32;
  __shared__ float w[kMaxSlots * G];
  __shared__ float red[NW][G];
  __shared__ float4 acc[kCombine];
  const int b = blockIdx.x / p.Hkv, kvh = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Head hd = *p.ws.head;
  const RowRec r = p.ws.row[b];
  // prefix slots: how many, their first, whether there are two a CTA, and where the row's
  // heads lie in them
  int n1 = 0, first1 = 0, step1 = 0, two1 = 0, off1 = 0, i1 = 0, rows1 = 0;
  if (r.group >= 0) {
    const GroupRec g = p.ws.grp[r.group];
    const int i = (b - g.row0) * G, pair = i / (2 * TILE), ii = i % (2 * TILE);
    const int item = kvh * g.npairs + pair, left = g.nrows * G - pair * 2 * TILE;
    const int a = g.off + item * g.nt * g.cost, c0 = a / hd.share;
    n1 = (a + (g.nt - 1) * g.cost) / hd.share - c0 + 1;
    const int second = ii >= TILE ? TILE : 0;               // of a pair's query tiles
    first1 = g.base + (c0 - g.cf + item) * g.rows + second;
    i1 = ii - second;
    rows1 = min(left - second, TILE);
    step1 = g.rows;
    two1 = left <= TILE;
    off1 = g.npairs == 1 ? left : TILE;
  }
  int n2 = 0, first2 = 0;                                   // the row's own slots
  if (r.nt > 0) {
    const int a = p.ws.cta[0].prefix_cost + r.off + kvh * hd.cost.own_cost(r.nt), c0 = a / hd.share;
    n2 = (a + hd.cost.own_begin(r.nt - 1)) / hd.share - c0 + 1;
    first2 = hd.suffix_base + (c0 + b * p.Hkv + kvh) * 2 * G;
  }
  const int m1 = n1 * (1 + two1), n = min(m1 + 2 * n2, kMaxSlots);
  auto slot = [&](int k) -> int {          // first row of slot k
    int s;
    if (k < m1) s = two1 ? first1 + (k >> 1) * step1 + (k & 1) * off1 : first1 + k * step1;
    else s = first2 + (k - m1) * G;
    return ETA_RANGE_IN_BOUNDS(s, s + (k < m1 ? rows1 : G), p.part_rows, p.status) ? s : 0;
  };
  auto row_of = [&](int k) -> int { return slot(k) + (k < m1 ? i1 : 0); };
  // a thread's elements (slot, head) all have the head tid % G
  auto over_threads = [&](float v, auto op) -> float {
#pragma unroll
    for (int x = 16; x >= G; x >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, x));
    if (lane < G) red[warp][lane] = v;
    __syncthreads();
    v = red[0][tid % G];
#pragma unroll
    for (int i = 1; i < NW; ++i) v = op(v, red[i][tid % G]);
    __syncthreads();
    return v;
  };
  const float2* ml = reinterpret_cast<const float2*>(p.ws.part_ml);
  constexpr int KEEP = 4;                   // elements a thread keeps (512 slots of 4 heads)
  float2 kept[KEEP];
  float mx = -INFINITY;
#pragma unroll
  for (int u = 0; u < KEEP; ++u) {
    const int x = tid + u * kCombine;
    kept[u] = x < n * G ? ml[row_of(x / G) + x % G] : make_float2(-INFINITY, 0.f);
    mx = fmaxf(mx, kept[u].x);
  }
  for (int x = tid + KEEP * kCombine; x < n * G; x += kCombine)
    mx = fmaxf(mx, ml[row_of(x / G) + x % G].x);
  mx = over_threads(mx, [](float a, float c) { return fmaxf(a, c); });
  float l = 0.f;
  auto weigh = [&](int x, float2 v) {
    const float e = mx == -INFINITY ? 0.f : expf(v.x - mx);
    w[x] = e;
    l = fmaf(e, v.y, l);
  };
#pragma unroll
  for (int u = 0; u < KEEP; ++u)
    if (tid + u * kCombine < n * G) weigh(tid + u * kCombine, kept[u]);
  for (int x = tid + KEEP * kCombine; x < n * G; x += kCombine)
    weigh(x, ml[row_of(x / G) + x % G]);
  l = over_threads(l, [](float a, float c) { return a + c; });
  const size_t head0 = (size_t)b * p.Hq + kvh * G;
  if (tid < G) {
    lse[head0 + tid] = l != 0.f ? mx + logf(l) : -INFINITY;   // NaN passes on
    red[0][tid] = l;
  }
  // head fastest: the G heads of 4 dims are side by side in a slot
  const int v = tid % VEC, gi = tid / VEC, h = v % G, vd = v / G;
  const float4* po = reinterpret_cast<const float4*>(p.ws.part_o);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = gi; k < n; k += NG) {
    const float4 x = k < m1 ? po[(size_t)slot(k) * (D / 4) + vd * rows1 + i1 + h]
                            : po[(size_t)slot(k) * (D / 4) + vd * G + h];
    const float e = w[k * G + h];
    if (e > 0.f) {                          // an empty slot's o was never written
      a.x = fmaf(e, x.x, a.x);
      a.y = fmaf(e, x.y, a.y);
      a.z = fmaf(e, x.z, a.z);
      a.w = fmaf(e, x.w, a.w);
    }
  }
  acc[tid] = a;
  __syncthreads();
  if (gi == 0) {
#pragma unroll
    for (int i = 1; i < NG; ++i) {
      const float4 y = acc[i * VEC + v];
      a.x += y.x;
      a.y += y.y;
      a.z += y.z;
      a.w += y.w;
    }
    const float L = red[0][h];
    if (L != 0.f) {
      a.x /= L;
      a.y /= L;
      a.z /= L;
      a.w /= L;
    } else {
      a = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    store4(o + (head0 + h) * D + vd * 4, a);
  }
}

// ------------------------------------------------------------------------- host side
struct WsOff {
  size_t head, grp, row, cta, ml, o, total;
  int part_rows;
};

inline WsOff ws_off(const eta_dims_t* d, int n_groups, int P) {
  // slots: at most 256 rows for every CTA and twice a group's own rows for every item,
  // and 2 G rows for every CTA and (row, KV head)
  const int G = d->Hq / d->Hkv;
  WsOff w;
  const size_t rows = (size_t)P * (2 * TILE + 2 * G) + 4 * (size_t)d->B * d->Hq;
  size_t x = 0;
  w.head = x; x += 256;
  w.grp = x;  x = align_up(x + (size_t)n_groups * sizeof(GroupRec), 256);
  w.row = x;  x = align_up(x + (size_t)d->B * sizeof(RowRec), 256);
  w.cta = x;  x = align_up(x + (size_t)P * sizeof(CtaRec), 256);
  w.ml = x;   x = align_up(x + rows * 8, 256);
  w.o = x;    x = align_up(x + rows * d->d * 4, 256);
  w.total = x;
  w.part_rows = (int)rows;
  return w;
}

inline int grid_size() { return std::max(sm_count(), 1); }

// Sizes whose costs fit 32-bit sums, and whose parts fit the combine's list.
inline eta_status_t check_sizes(const eta_dims_t* d, int32_t n_groups, int P) {
  if (n_groups < 1 || n_groups > d->B) return ETA_ERR_INVALID_ARG;
  const uint64_t tiles = ((uint64_t)d->T_max + TILE - 1) / TILE;
  if (16 * tiles * d->B * d->Hkv >= (1ull << 31)) return ETA_ERR_UNSUPPORTED;
  if ((uint64_t)P * 528 + 4ull * d->B * d->Hq >= (1ull << 31)) return ETA_ERR_UNSUPPORTED;
  if (4 * P > kMaxSlots) return ETA_ERR_UNSUPPORTED;
  return ETA_OK;
}

template <int D, int GATE, int NS>
eta_status_t launch_attend(const CUtensorMap& mq, const CUtensorMap& mq1, const CUtensorMap& mk,
                           const CUtensorMap& mv, const AttendParams& a, int P, cudaStream_t s) {
  if (!set_smem_once<shared_attend_kernel<D, GATE, NS>>(Cfg<D>::SMEM)) return ETA_ERR_CUDA;
  return launch_k(shared_attend_kernel<D, GATE, NS>, dim3(P), dim3(NT), Cfg<D>::SMEM, s, mq, mq1,
                  mk, mv, a);
}

template <int D>
eta_status_t launch_attend_d(int gate, bool two, const CUtensorMap& mq, const CUtensorMap& mq1,
                             const CUtensorMap& mk, const CUtensorMap& mv, const AttendParams& a,
                             int P, cudaStream_t s) {
  switch (gate * 2 + (two ? 1 : 0)) {
    case 0: return launch_attend<D, NONE, 1>(mq, mq1, mk, mv, a, P, s);
    case 1: return launch_attend<D, NONE, 3>(mq, mq1, mk, mv, a, P, s);
    case 2: return launch_attend<D, HARD, 1>(mq, mq1, mk, mv, a, P, s);
    case 3: return launch_attend<D, HARD, 3>(mq, mq1, mk, mv, a, P, s);
    case 4: return launch_attend<D, SOFT, 1>(mq, mq1, mk, mv, a, P, s);
    default: return launch_attend<D, SOFT, 3>(mq, mq1, mk, mv, a, P, s);
  }
}

template <int G>
eta_status_t launch_combine(const eta_dims_t* d, bool f32, const AttendParams& a, void* o,
                            float* lse, cudaStream_t s) {
  const dim3 grid(d->B * d->Hkv), block(kCombine);
  if (f32)
    return d->d == 64 ? launch_k(shared_combine_kernel<64, G, float>, grid, block, 0, s, a,
                                 static_cast<float*>(o), lse)
                      : launch_k(shared_combine_kernel<128, G, float>, grid, block, 0, s, a,
                                 static_cast<float*>(o), lse);
  return d->d == 64 ? launch_k(shared_combine_kernel<64, G, __nv_bfloat16>, grid, block, 0, s, a,
                               static_cast<__nv_bfloat16*>(o), lse)
                    : launch_k(shared_combine_kernel<128, G, __nv_bfloat16>, grid, block, 0, s, a,
                               static_cast<__nv_bfloat16*>(o), lse);
}

// q [B, Hq, d] as (dim, head, row); box 64 x G x rows, 128-byte swizzle.
inline bool make_map_q(CUtensorMap* m, const void* q, const eta_dims_t* d, int rows) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t gdim[3] = {(cuuint64_t)d->d, (cuuint64_t)d->Hq, (cuuint64_t)d->B};
  cuuint64_t gstride[2] = {(cuuint64_t)d->d * 2, (cuuint64_t)d->Hq * d->d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)(d->Hq / d->Hkv), (cuuint32_t)rows};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), gdim, gstride, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace sd
}  // namespace eta

using namespace eta;

extern "C" size_t eta_shared_decode_workspace_size(const eta_dims_t* dims, int32_t n_groups) {
  if (check_dims(dims) != ETA_OK) return 0;
  const int P = sd::grid_size();
  if (sd::check_sizes(dims, n_groups, P) != ETA_OK) return 0;
  return sd::ws_off(dims, n_groups, P).total;
}

extern "C" eta_status_t eta_shared_decode(const eta_dims_t* dims, int32_t n_pages,
                                          int32_t n_groups, const eta_bf16_t* q,
                                          const float* tau, const eta_bf16_t* K_pool,
                                          const eta_bf16_t* V_pool, const int32_t* table,
                                          const int32_t* lengths, const int32_t* group_off,
                                          const int32_t* prefix_len, float T, float scale,
                                          eta_out_format_t o_format, void* o, float* lse,
                                          void* ws, size_t ws_bytes, int32_t* dev_status,
                                          void* stream) {
  eta_status_t st = check_pool(dims, n_pages);
  if (st != ETA_OK) return st;
  const int P = sd::grid_size();
  if ((st = sd::check_sizes(dims, n_groups, P)) != ETA_OK) return st;
  if (!q || !K_pool || !V_pool || !table || !lengths || !group_off || !prefix_len || !o || !lse)
    return ETA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(K_pool) || !aligned16(V_pool) || !aligned16(o))
    return ETA_ERR_INVALID_ARG;
  if (o_format != ETA_OUT_F32 && o_format != ETA_OUT_BF16) return ETA_ERR_INVALID_ARG;
  if (tau && (!(T >= 0.f) || isinf(T))) return ETA_ERR_INVALID_ARG;
  if (!(scale >= 0.f) || isinf(scale)) return ETA_ERR_INVALID_ARG;   // the gate divides by it
  const sd::WsOff L = sd::ws_off(dims, n_groups, P);
  if (!ws || ws_bytes < L.total || !aligned16(ws)) return ETA_ERR_WORKSPACE;
  if (scale == 0.f) scale = 1.f / sqrtf((float)dims->d);

  const int G = dims->Hq / dims->Hkv;
  CUtensorMap mq, mq1, mk, mv;
  const uint64_t kv_rows = (uint64_t)n_pages * dims->Hkv * dims->blk;
  if (!sd::make_map_q(&mq, q, dims, sd::TILE / G) || !sd::make_map_q(&mq1, q, dims, 1) ||
      !make_map(&mk, K_pool, kv_rows, sd::SUB, dims->d) ||
      !make_map(&mv, V_pool, kv_rows, sd::SUB, dims->d))
    return ETA_ERR_CUDA;
  char* w = static_cast<char*>(ws);
  sd::Ws wp;
  wp.head = reinterpret_cast<sd::Head*>(w + L.head);
  wp.grp = reinterpret_cast<sd::GroupRec*>(w + L.grp);
  wp.row = reinterpret_cast<sd::RowRec*>(w + L.row);
  wp.cta = reinterpret_cast<sd::CtaRec*>(w + L.cta);
  wp.part_ml = reinterpret_cast<float*>(w + L.ml);
  wp.part_o = reinterpret_cast<float*>(w + L.o);
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  sd::PlanParams pp;
  pp.B = dims->B; pp.Hkv = dims->Hkv; pp.G = G; pp.NB = num_blocks(dims); pp.blk = dims->blk;
  pp.n_groups = n_groups; pp.n_pages = n_pages; pp.P = P; pp.lengths = lengths; pp.group_off = group_off;
  pp.prefix_len = prefix_len; pp.table = table; pp.ws = wp; pp.status = dev_status;
  st = launch_k(sd::shared_plan_kernel, dim3(1), dim3(sd::kPlan), 0, s, pp);
  if (st != ETA_OK) return st;

  sd::AttendParams a;
  a.B = dims->B; a.Hq = dims->Hq; a.Hkv = dims->Hkv; a.G = G; a.NB = pp.NB; a.blk = dims->blk;
  a.n_pages = n_pages; a.n_groups = n_groups; a.scale = scale;
  a.invT = T > 0.f ? inverse_temperature(T) : 0.f;
  a.tau = tau; a.table = table; a.lengths = lengths; a.ws = wp; a.part_rows = L.part_rows;
  a.status = dev_status;
  const int gate = !tau ? sd::NONE : T == 0.f ? sd::HARD : sd::SOFT;
  const bool two = o_format == ETA_OUT_F32, d64 = dims->d == 64;
  st = d64 ? sd::launch_attend_d<64>(gate, two, mq, mq1, mk, mv, a, P, s)
           : sd::launch_attend_d<128>(gate, two, mq, mq1, mk, mv, a, P, s);
  if (st != ETA_OK) return st;

  switch (G) {
    case 1: return sd::launch_combine<1>(dims, two, a, o, lse, s);
    case 2: return sd::launch_combine<2>(dims, two, a, o, lse, s);
    case 4: return sd::launch_combine<4>(dims, two, a, o, lse, s);
    default: return sd::launch_combine<8>(dims, two, a, o, lse, s);
  }
}
