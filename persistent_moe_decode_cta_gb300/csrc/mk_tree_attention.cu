// Attention of several nodes per sequence over the paged cache and one another.
//
//   out_i = sum_j 2^(c q_i.k_j - m_i) v_j / sum_j 2^(c q_i.k_j - m_i),   c = scale / ln 2
// in one pass over the keys, with the running maximum m_i and the running sum in fp32.
//
// A row is a (node, query head) pair of one KV head: row r of a tile is node r / gs, head
// r % gs, so that the gs heads of a group share every key that is read.  A tile has 128
// rows, the M of one tcgen05.mma; S = Q K^T and O += P V both run on the tensor cores with
// accumulators in tensor memory, P goes back there as bf16 (A operand), and the thread that
// owns a row (lane) keeps its maximum and sum.  (P and V of one product have one type, and V is
// bf16: each weight is rounded to 8 bits, in the sum it keeps its 24.  Against float64 the results are
// 0.0021 to 0.0024 off, relative; their own rounding alone is 0.0017.)  Keys come in blocks of 128 (8 pages), each
// page by its own tensor-map copy, into a ring shared by K and V.
//
// Two softmax warpgroups ("streams") alternate so that one's exponentials run beside the
// other's products.  Up to 128 rows per KV head both streams work on the same rows, on
// even and odd key blocks, and are merged at the end (TWO = false); with more rows each
// stream has a tile of its own and both use every key block that is loaded (TWO = true),
// which halves the key traffic where it would exceed what L2 delivers.
//
// One thread issues all products.  TWO = true is bound by them: P V of a block and S of the
// stream's next one go out behind one wait (32 products of 64 cycles a pair of blocks; the queue
// does not cover the 60 to 75 cycles of each wait).  TWO = false is bound by the copies: a
// stream takes a block in two halves with an S/P buffer each, and S of a block is computed as soon
// as its K is there, whatever the softmax is at, so that the slots of the ring are free again early
// (16 nodes at 32K of 8 sequences: 106 us, with whole blocks 122).
//
// Keys that a row does not see get a score of -infinity.  Blocks with such keys have their V
// cleaned in shared memory by two further warps (rows past the end and values that are not
// finite become zero, since 0 * NaN would reach every row); what was dropped is added with plain
// loads at the end, for the rows that do see it.
//
// The work is a list of units, one per (sequence, tile group, KV head, key block), cut into
// equal runs, one per CTA: ragged batches and single long sequences fill all SMs alike.  An item, the
// keys of one KV head for one tile group, counts for six units more: a run that starts one pays for its
// queries, the empty pipeline and one more result.  (Without them the 31 of 152 CTAs whose run holds a
// border of 8 sequences' items end 8 us after the others: 58.4 us against 51.3 for 16 nodes of 8 ragged
// sequences, 18.6 against 15.7 for one node at 8K, 332 against 152 for a prompt of 4096, whose first items
// are short, when that was changed.  3 to 8 are within 3% of one another.)  (Up
// to 8 tile groups form a team instead: each run is walked by one CTA per group at the same
// time, so that the keys come from HBM once and from L2 for the others.)  A run that covers
// only part of an item's keys leaves (O, m, sum) in the workspace and a second kernel joins
// the parts in order of their keys; at most a run's first and last item are such.
//
// Measured, 32 query heads and 4 KV heads of 128: 16 nodes at 32K of 8 sequences 97 us (5.6 TB/s), 64 nodes
// 198 us (1.39 PFLOP/s), 2001 nodes of a chunk at 8K 224 us (1.34 PFLOP/s), one node at 8K of one sequence
// 16.7 us, 8 nodes at 2K of the small model 12.7 us (latencies).
#include "mk_ops.cuh"

#include <type_traits>

namespace mk {
namespace {

constexpr int kBlk = 128;               // keys of a block
constexpr int kTreeThreads = 384;       // two softmax warpgroups; a copy, a product and two cleaning warps
constexpr int kCleaners = 64;
constexpr int kTmemS = 0, kTmemO = 256;  // columns: S/P of the streams at 0 and 128, O at 256 and 384
constexpr float kRescale = 8.f;         // the maximum may lag by 2^8 before O is rescaled

// Shared-memory layout of a tile of 128 rows: groups of 8 rows, of each group the spans one
// behind the other, of each span 8 swizzled lines.  A page (16 rows) is then one contiguous
// piece that one copy fills, and a group is kGroup bytes from the next in every page.
template <int HD>
struct TreeCfg {
  static constexpr int kSpan = HD == 32 ? 64 : 128;        // swizzle span in bytes
  static constexpr int kHalves = HD * 2 / kSpan;           // spans per row
  static constexpr int kGroup = 8 * HD * 2;                // 8 rows
  static constexpr int kTile = kBlk * HD * 2;              // 128 rows
  static constexpr int kSlots = HD == 128 ? 7 : 10;        // query tiles and ring stages together
  // the row that 16-byte piece i of a tile belongs to
  __host__ __device__ static constexpr int row_of(int i) { return i / (kGroup / 16) * 8 + i / (kSpan / 16) % 8; }
  // byte offset of column 16 kk of a tile's first row group
  __host__ __device__ static constexpr int column16(int kk) { return (kk * 32 / kSpan) * (8 * kSpan) + (kk * 32) % kSpan; }
};

// ------------------------------------------------------------------ work list

struct Item {          // one (sequence, KV head, tile group) and the blocks of this run
  int b, kvh, tp;
  int len, cnt;        // cached tokens, nodes
  int kstart, end;     // its keys: [kstart, end)
  int nblk;            // their blocks
  int ja, jb;          // blocks of this run
  int unit0;           // global index of its first unit
};

struct SeqShape {
  int len, cnt;
};

// Length and node count of a sequence; an invalid one gets no nodes.
__device__ __forceinline__ SeqShape seq_shape(const TreeParams& p, int b, bool record) {
  SeqShape s;
  s.len = op_ld(p.c.seq_lens + b);
  s.cnt = p.a.counts ? op_ld(p.a.counts + b) : p.a.n_nodes;
  if (s.len < 0 || s.cnt > p.a.n_nodes || (long long)s.len + s.cnt > 16ll * p.c.max_pages) {
    if (record) op_error(p.a.status, MK_ERR_INVALID, b, s.cnt, s.len);
    s.cnt = 0;
  }
  if (s.cnt < 0) s.cnt = 0;
  return s;
}

__device__ __forceinline__ int nodes_per_group(const TreeParams& p) { return p.npt * (p.two ? 2 : 1); }

// An entry of the work list: the tile groups [tp, tp + team) of sequence b.  All of them
// start at the same key; with the causal chain each ends at its own last node.  A window starts
// at the earliest key that any of their nodes may see (on a page boundary).
struct Entry {
  int b, tp;           // first tile group
  SeqShape s;
  int kstart, nblk;    // blocks of the longest
  int units;           // per KV head: the blocks and kItemUnits
};

// end of the keys of tile group tp (0 if it has no nodes)
__device__ __forceinline__ int group_end(const TreeParams& p, const SeqShape& s, int tp) {
  const int per = nodes_per_group(p), first = tp * per;
  if (first >= s.cnt) return 0;
  return s.len + (p.a.mask ? s.cnt : min(s.cnt, first + per));
}

__device__ __forceinline__ Entry make_entry(const TreeParams& p, int e, bool record) {
  Entry x;
  x.b = p.groups == 1 ? e : e / p.groups;
  x.tp = (e - x.b * p.groups) * p.team;
  x.s = seq_shape(p, x.b, record);
  x.kstart = x.nblk = x.units = 0;
  const int per = nodes_per_group(p), first = x.tp * per;
  if (first >= x.s.cnt) return x;
  const int end = x.s.len + (p.a.mask ? x.s.cnt : min(x.s.cnt, first + p.team * per));  // of its last group with nodes
  if (p.a.window > 0) {
    const int pos = x.s.len + (p.a.mask || p.a.positions ? 0 : first);  // the earliest position of its nodes
    x.kstart = max(0, pos - p.a.window + 1) & ~(kOpPage - 1);
  }
  x.nblk = (end - x.kstart + kBlk - 1) / kBlk;
  x.units = x.nblk + kItemUnits;
  return x;
}

__device__ __forceinline__ int num_entries(const TreeParams& p) { return p.c.batch * p.groups; }

constexpr int kScan = 128;  // threads that add up the work list
constexpr int kJoinThreads = 256;

// Prefix sums of the entries' units: thread i < kScan owns entries [i * chunk, (i + 1) *
// chunk), pre[i] is the number of units before them, pre[kScan] that of all.
__device__ void scan_units(const TreeParams& p, int* pre, int* warp_sums, bool record) {
  const int E = num_entries(p), chunk = (E + kScan - 1) / kScan;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = 0;
  if (threadIdx.x < kScan)
    for (int e = (int)threadIdx.x * chunk; e < min(E, ((int)threadIdx.x + 1) * chunk); ++e)
      x += make_entry(p, e, record).units * p.c.n_kv_heads;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31 && w < kScan / 32) warp_sums[w] = x;
  __syncthreads();
  if (threadIdx.x < kScan) {
    for (int i = 0; i < w; ++i) x += warp_sums[i];
    pre[threadIdx.x + 1] = x;
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}

// Units of a run: run g, of team g, is [g * n, (g + 1) * n) up to U, so the parts of an item are those
// of consecutive teams.  (The longest run is what an even split would have, and the owner of a unit is
// one division away.  One tile: at least two blocks a run, since its two streams take one each.)
__device__ __forceinline__ int run_units(const TreeParams& p, int U) { return max((U + p.teams - 1) / p.teams, p.two ? 1 : 2); }

// Walks the items of a run for tile group `member` of its team.
struct Run {
  int u, u1, member;
  int e, first;        // the entry that unit u lies in or behind, and its first unit
  Entry x;
  Item it;

  __device__ __forceinline__ void start(const TreeParams& p, const int* pre) {
    int lo = -1;  // the last chunk that starts at or before u (so it has units)
#pragma unroll
    for (int i = 0; i < kScan; i += 32) lo += __popc(__ballot_sync(0xffffffffu, pre[i + (threadIdx.x & 31)] <= u));
    e = lo * ((num_entries(p) + kScan - 1) / kScan);
    first = pre[lo];
    x = make_entry(p, e, false);
  }
  // (up to 32 entries: lane i knows the units before entry i)
  __device__ __forceinline__ void start_short(const TreeParams& p, int before) {
    e = __popc(__ballot_sync(0xffffffffu, before <= u)) - 1;
    first = __shfl_sync(0xffffffffu, before, e);
    x = make_entry(p, e, false);
  }
  // The next item with blocks of this group in the run.  (One copy for all roles: an inlined
  // one per role, rarely run, costs thousands of cycles of instruction fetches each time.)
  __device__ __noinline__ bool next(const TreeParams& p) {
    while (u < u1) {
      while (u >= first + x.units * p.c.n_kv_heads) {
        first += x.units * p.c.n_kv_heads;
        x = make_entry(p, ++e, false);
      }
      it.b = x.b;
      it.tp = x.tp + member;
      it.len = x.s.len;
      it.cnt = x.s.cnt;
      it.kvh = (u - first) / x.units;
      it.unit0 = first + it.kvh * x.units;
      it.kstart = x.kstart;
      it.end = group_end(p, x.s, it.tp);
      it.nblk = max(0, it.end - it.kstart + kBlk - 1) / kBlk;
      const int start = u - it.unit0, stop = min(x.units, start + (u1 - u));
      u = it.unit0 + stop;
      it.ja = max(0, start - kItemUnits);
      it.jb = min(stop - kItemUnits, it.nblk);
      if (it.ja < it.jb) return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ what a row sees

struct Row {
  int node;     // -1: not a row of the call
  int pos;      // its position (clamped to [len, len + cnt - 1])
  int lo;       // the first position inside its window
  const int32_t* mask;
};

__device__ __forceinline__ Row make_row(const TreeParams& p, const Item& it, int node) {
  Row r;
  r.node = node;
  r.pos = it.len;
  r.lo = INT_MIN;
  r.mask = nullptr;
  if (node < 0) return r;
  const long long at = (long long)it.b * p.a.n_nodes + node;
  r.pos = it.len + node;
  if (p.a.window > 0) {
    if (p.a.positions) r.pos = min(max(op_ld(p.a.positions + at), it.len), it.len + it.cnt - 1);
    r.lo = r.pos - p.a.window + 1;
  }
  if (p.a.mask) r.mask = p.a.mask + at * p.words;
  return r;
}

// Bit i: the row sees key kb + i (32 keys).
__device__ __noinline__ uint32_t sees32(const TreeParams& p, const Item& it, const Row& r, int kb) {
  if (r.node < 0) return 0;
  uint32_t bits = 0;
  if (kb < it.len) {  // cached keys [max(lo, kb), min(len, kb + 32))
    const int a = r.lo > kb ? r.lo - kb : 0, e = min(it.len - kb, 32);
    if (a < e) bits = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & (0xffffffffu << a);
  }
  if (kb + 32 > it.len) {  // nodes a0 .. a0 + 31 (a0 > -32)
    const int a0 = kb - it.len;
    uint32_t nb;
    if (r.mask) {
      const int w = a0 >> 5, sh = a0 & 31;  // (floor)
      const uint32_t x = w >= 0 && w < p.words ? (uint32_t)op_ld(r.mask + w) : 0u;
      const uint32_t y = sh && w + 1 < p.words ? (uint32_t)op_ld(r.mask + w + 1) : 0u;
      nb = __funnelshift_r(x, y, sh);
    } else {
      const int e = r.node - a0 + 1;  // nodes 0..node
      nb = e <= 0 ? 0u : e >= 32 ? 0xffffffffu : (1u << e) - 1u;
    }
    const int e = it.cnt - a0;
    if (e < 32) nb &= e <= 0 ? 0u : (1u << e) - 1u;
    if (a0 < 0) nb &= 0xffffffffu << -a0;
    if (r.lo > it.len && nb) {  // the window reaches past the cache: look at the nodes' positions
      for (uint32_t m = nb; m; m &= m - 1) {
        const int i = __ffs(m) - 1, a = a0 + i;
        int pa = it.len + a;
        if (p.a.positions)
          pa = min(max(op_ld(p.a.positions + (long long)it.b * p.a.n_nodes + a), it.len), it.len + it.cnt - 1);
        if (pa < r.lo) nb &= ~(1u << i);
      }
    }
    bits |= nb;
  }
  return bits;
}

// Whether some row of the item may not see some key of the block at k0, or the block has
// keys past the end: its scores are masked and its V checked.
__device__ __forceinline__ bool masked_block(const TreeParams& p, const Item& it, int k0) {
  const int per = nodes_per_group(p);
  // keys below `open` are seen by all rows, but for a window that leaves their slots behind (with
  // positions of their own, nodes may be behind it whatever their slots are)
  const bool chain = !p.a.mask && !(p.a.window > 0 && p.a.positions);
  const int open = it.len + (chain ? it.tp * per + 1 : 0);
  if (k0 + kBlk > open) return true;
  if (p.a.window > 0) {
    const int last = p.a.mask || p.a.positions ? it.cnt : min(it.cnt, (it.tp + 1) * per);
    return k0 < it.len + last - p.a.window;  // the latest row's window starts inside or behind
  }
  return false;
}

// ------------------------------------------------------------------ shared memory

constexpr int kMaxStages = 9;
struct TreeShared {
  uint32_t tmem;
  int abort;
  int bad_v;             // a masked block held a V that is not finite
  Run runs[4];           // of the copy, product and cleaning warps
  float2 ml[2][kBlk];    // the streams' (m, sum) for the merge
  unsigned long long bars[3 * kMaxStages + 17];
};

template <int HD>
struct TreeSmem {
  static constexpr int kBytes = TreeCfg<HD>::kSlots * TreeCfg<HD>::kTile + (int)sizeof(TreeShared);
  static_assert(kBytes <= 232448, "exceeds the 227 KB per-block shared memory limit");
};

// Key block i of the CTA's run (i modulo the ring's slots) has barriers of its own for its K and
// its V: whoever waits for one has seen, or knows done, its previous use, so that the parity
// of a phase says which one it is.  (A slot's fills alternate between K and V when the number
// of slots is odd, and nobody sees them all but the producer.)
struct Bars {
  uint32_t base;
  __device__ __forceinline__ uint32_t kfull(uint32_t i) const { return base + 8 * i; }                     // copied
  __device__ __forceinline__ uint32_t vfull(uint32_t i) const { return base + 8 * (kMaxStages + i); }
  __device__ __forceinline__ uint32_t empty(uint32_t s) const { return base + 8 * (2 * kMaxStages + s); }  // slot s read
  __device__ __forceinline__ uint32_t one(int i) const { return base + 8 * (3 * kMaxStages + i); }
  __device__ __forceinline__ uint32_t qfull() const { return one(0); }
  __device__ __forceinline__ uint32_t qempty() const { return one(1); }
  __device__ __forceinline__ uint32_t meet() const { return one(2); }
  // (TWO = false: per half h of a block)
  __device__ __forceinline__ uint32_t sfull(uint32_t st, uint32_t h) const { return one(3 + 2 * st + h); }   // S computed
  __device__ __forceinline__ uint32_t pready(uint32_t st, uint32_t h) const { return one(7 + 2 * st + h); }  // P written (h = 0: V fit for use)
  __device__ __forceinline__ uint32_t pvdone(uint32_t st, uint32_t h) const { return one(11 + 2 * st + h); } // its P V (TWO = false)
  __device__ __forceinline__ uint32_t ofull(uint32_t st) const { return one(15 + st); }                      // an item's last P V
};

__device__ __forceinline__ bool nonfinite2(uint32_t u) {
  return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t drop_nonfinite2(uint32_t u) {
  if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) u &= 0x0000ffffu;
  return u;
}

// Threads t of NT: in the landed V block at `stage`, rows from `live` on become zero and
// values that are not finite are dropped (and reported): a weight of zero times such a value
// would otherwise reach rows that do not see the key.  Sixteen bytes at a time, eight loads
// together; an exponent of all ones carries into the sign's place when one is added to it.
template <int HD, int NT>
__device__ __noinline__ void clean_v(uint8_t* stage, int live, int t, int* bad) {
  using C = TreeCfg<HD>;
  constexpr int kVecs = C::kTile / 16 / NT, kBatch = 8;
  static_assert(kVecs % kBatch == 0, "batches");
  uint4* const at = reinterpret_cast<uint4*>(stage) + t;
#pragma unroll 1
  for (int i0 = 0; i0 < kVecs; i0 += kBatch) {
    uint4 x[kBatch];
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) x[i] = at[(i0 + i) * NT];
    auto carry = [](uint32_t u) { return (u & 0x7f807f80u) + 0x00800080u; };
#pragma unroll
    for (int i = 0; i < kBatch; ++i) any |= carry(x[i].x) | carry(x[i].y) | carry(x[i].z) | carry(x[i].w);
    const bool past = C::row_of((i0 + kBatch - 1) * NT + NT - 1) >= live;  // (rows ascend along the tile)
    if (!past && !(any & 0x80008000u)) continue;
#pragma unroll 1
    for (int i = 0; i < kBatch; ++i) {
      uint4 y = at[(i0 + i) * NT];
      if (C::row_of((i0 + i) * NT + t) >= live) {
        y = make_uint4(0, 0, 0, 0);
      } else if (nonfinite2(y.x) || nonfinite2(y.y) || nonfinite2(y.z) || nonfinite2(y.w)) {
        y = make_uint4(drop_nonfinite2(y.x), drop_nonfinite2(y.y), drop_nonfinite2(y.z), drop_nonfinite2(y.w));
        *reinterpret_cast<volatile int*>(bad) = 1;
      } else {
        continue;
      }
      at[(i0 + i) * NT] = y;
    }
  }
}

__device__ __forceinline__ int page_of(const TreeParams& p, int b, int key) {
  const int page = op_ld(p.c.page_table + (long long)b * p.c.max_pages + key / kOpPage);
  return page >= 0 && page < p.c.n_pages ? page : 0;
}

// What clean_v dropped from columns [c0, c1) of a row: p_j * v_j of the keys that the row sees, added
// to the stored values (in any order and precision: each is an infinity or NaN, and so is the sum).
// Only after a masked block held such values (never with finite caches): plain loads.
template <int HD>
__device__ __noinline__ void put_nonfinite(const TreeParams& p, const Item& it, const Row& r, int head, float m, float inv, int c0,
                                           int c1, uint16_t* dst, float4* part) {
  const uint16_t* q = static_cast<const uint16_t*>(p.a.q) + it.b * p.a.q_stride[0] + r.node * p.a.q_stride[1] + head * p.a.q_stride[2];
  const uint16_t* K = static_cast<const uint16_t*>(p.c.k);
  const uint16_t* V = static_cast<const uint16_t*>(p.c.v);
  for (int j = it.ja; j < it.jb; ++j) {
    const int k0 = it.kstart + j * kBlk;
    if (!masked_block(p, it, k0)) continue;
    for (int w = 0; w < kBlk / 32; ++w) {
      for (uint32_t bits = sees32(p, it, r, k0 + 32 * w); bits; bits &= bits - 1) {
        const int key = k0 + 32 * w + __ffs(bits) - 1;
        const long long at = (((long long)page_of(p, it.b, key) * p.c.n_kv_heads + it.kvh) * kOpPage + key % kOpPage) * HD;
        uint32_t any = 0;
#pragma unroll
        for (int c = 0; c < HD; c += 8) {
          const uint4 v = op_ld16(V + at + c);
          any |= (uint32_t)(nonfinite2(v.x) || nonfinite2(v.y) || nonfinite2(v.z) || nonfinite2(v.w)) << (c / 8);
        }
        if (!any) continue;
        float s = 0.f;
        for (int d = 0; d < HD; d += 8) {
          const uint4 a = op_ld16(q + d), b = op_ld16(K + at + d);
          const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_f2(x[i]), g = bf16x2_to_f2(y[i]);
            s += f.x * g.x + f.y * g.y;
          }
        }
        const float weight = ex2(s * p.scale_log2 - m);
        for (int c = c0; c < c1; ++c) {
          if (!(any >> (c / 8) & 1u)) continue;
          const float v = bf16_to_f(V[at + c]);
          if (fabsf(v) <= 3.4e38f) continue;
          if (dst) {
            volatile uint16_t* o = dst + c;
            *o = to_bf16(bf16_to_f(*o) + weight * v * inv);
          } else {
            volatile float* o = reinterpret_cast<float*>(part + (c / 4) * kBlk) + c % 4;
            *o = *o + weight * v;
          }
        }
      }
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Store 16 columns of a row: the result (one 32-byte sector), or the row's part of it (a
// float4 per 4 columns, rows side by side).
__device__ __forceinline__ void put16(const float (&o)[16], bool whole, float inv, uint16_t* dst, float4* part, int c) {
  if (whole) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {  // (a lane's row is a line of its own: one access, not two)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) __stcg(part + (c / 4 + i) * kBlk, make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
  }
}

template <int HD, bool TWO>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tq,
                const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using C = TreeCfg<HD>;
  constexpr uint32_t kStages = C::kSlots - (TWO ? 2 : 1);
  constexpr int kParts = TWO ? 2 : 1;  // halves of a block that a softmax step takes
  static_assert(kStages <= kMaxStages, "barriers");
  // (no static shared memory: the tiles start at its first byte, which is aligned to 1024)
  extern __shared__ __align__(1024) uint8_t raw[];
  TreeShared& sh = *reinterpret_cast<TreeShared*>(raw + C::kSlots * C::kTile);
  const uint32_t base = smem_u32(raw);
  if (base & 1023u) {
    pdl_wait();
    if (threadIdx.x == 0) op_error(p.a.status, MK_ERR_UNSUPPORTED, -1, (int)base, 0);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.table[kScan] = 0;
    return;
  }
  const uint32_t q_s = base, ring = base + (TWO ? 2 : 1) * C::kTile;
  uint8_t* const ring_g = raw + (ring - base);
  const Bars bars{smem_u32(sh.bars)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &sh.abort;

  if (warp == 8 && lane < 3) {
    const CUtensorMap* tm = lane == 0 ? &tk : lane == 1 ? &tv : &tq;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
  }
  if (warp == 11) tmem_alloc(smem_u32(&sh.tmem), 512);
  if (threadIdx.x == 128) {
    sh.abort = 0;
    sh.bad_v = 0;
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(bars.kfull(s), 1);
      mbar_init(bars.vfull(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    mbar_init(bars.qfull(), 1);
    mbar_init(bars.qempty(), 1);
    mbar_init(bars.meet(), 256);
    for (uint32_t st = 0; st < 2; ++st) {
      mbar_init(bars.ofull(st), 1);
      for (uint32_t h = 0; h < 2; ++h) {
        mbar_init(bars.sfull(st, h), 1);
        mbar_init(bars.pvdone(st, h), 1);
        mbar_init(bars.pready(st, h), h ? 128 : 128 + kCleaners);
      }
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sh.tmem);
  pdl_wait();
  pdl_trigger();
  // The units before each entry.  Up to 32 entries every warp adds them up by itself, without a barrier.
  const int E = num_entries(p);
  int* const pre = reinterpret_cast<int*>(raw);  // (where the queries go afterwards)
  int U, before = 0;
  if (E <= 32) {
    int own = 0;
    if (lane < E) own = make_entry(p, lane, blockIdx.x == 0 && warp == 0).units * p.c.n_kv_heads;
    U = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, U, o);
      if (lane >= o) U += y;
    }
    before = U - own;
    U = __shfl_sync(0xffffffffu, U, 31);
  } else {
    scan_units(p, pre, pre + kScan + 1, blockIdx.x == 0);
    if (blockIdx.x == 0 && threadIdx.x <= kScan && E > kJoinThreads) p.table[threadIdx.x] = pre[threadIdx.x];
    U = pre[kScan];
  }
  const int n = run_units(p, U);
  const int team = p.team == 1 ? (int)blockIdx.x : (int)blockIdx.x / p.team;
  if (team >= p.teams || team * n >= U) {  // (the whole CTA)
    if (warp == 11) tmem_dealloc(tmem, 512);
    return;
  }
  Run begin;
  begin.u = team * n;
  begin.u1 = min(U, begin.u + n);
  begin.member = (int)blockIdx.x - team * p.team;
  if (E <= 32) {
    begin.start_short(p, before);
  } else {
    begin.start(p, pre);
    fence_proxy_async_smem();
    __syncthreads();
  }
  const int u0 = begin.u;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax streams
    const uint32_t st = (uint32_t)warp >> 2;        // 0 or 1
    const int row = (int)threadIdx.x & 127;         // = lane of tensor memory
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t tS = tmem + kTmemS + 128 * st + lanes;
    const uint32_t tO = tmem + kTmemO + lanes;      // of stream 0; stream 1's is 128 columns on
    uint32_t ns = 0, nm = 0;                        // blocks of the stream, meetings
    uint32_t no[2] = {0, 0};                        // items of the streams
    bool ok = true;
    auto meet = [&]() -> bool {                     // all 256 threads of the two streams
      mbar_arrive(bars.meet());
      return op_wait(bars.meet(), nm++ & 1, abort, p.a.status, 7);
    };
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    Run run = begin;
    while (ok && uniform(run.next(p))) {
      const Item& it = run.it;
      const int nb = (int)uniform(it.jb - it.ja);
      const int tile = TWO ? (int)st : 0;
      const int node_in = row / p.gs;
      int node = it.tp * nodes_per_group(p) + tile * p.npt + node_in;
      if (node_in >= p.npt || node >= it.cnt) node = -1;
      const Row r = make_row(p, it, node);
      const bool warp_live = __any_sync(0xffffffffu, node >= 0);
      float m = -INFINITY, l = 0.f;
      const int b0 = TWO ? 0 : (int)st;
      for (int blk = b0; ok && blk < nb; blk += TWO ? 1 : 2) {
        const int k0 = it.kstart + (it.ja + blk) * kBlk;
        const bool masked = uniform(masked_block(p, it, k0));
#pragma unroll 1
        for (uint32_t h = 0; h < 2 / kParts; ++h) {
          constexpr int kW = kBlk / 2 * kParts;  // keys of a step
          uint32_t vis[kW / 32];
          if (masked) {
#pragma unroll
            for (int w = 0; w < kW / 32; ++w) vis[w] = sees32(p, it, r, k0 + kW * (int)h + 32 * w);
          }
          if (!(ok = op_wait(bars.sfull(st, h), ns & 1, abort, p.a.status, 9))) break;
          tc_fence_after();
          if (warp_live) {
            const uint32_t tSh = tS + kW * h;
            uint32_t s[kW];
#pragma unroll
            for (int i = 0; i < kW / 32; ++i) tmem_ld32(tSh + 32 * i, s + 32 * i);
#pragma unroll
            for (int i = 0; i < kW / 32; ++i) tmem_wait32(s + 32 * i);
            if (masked) {
#pragma unroll
              for (int i = 0; i < kW; ++i)
                if (!(vis[i >> 5] >> (i & 31) & 1u)) s[i] = 0xff800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kW; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
            const float mnew = fmaxf(m, max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * p.scale_log2);
            const bool grow = node >= 0 && mnew > m + kRescale;  // (also the first finite maximum)
            if (__any_sync(0xffffffffu, grow)) {
              const float f = mnew == m ? 1.f : ex2(m - mnew);
              if (blk != b0 || h) {
                // once the last P V has ended (TWO: S came after it)
                if (!TWO && !(ok = op_wait(bars.pvdone(st, h ^ 1), (ns - (h ^ 1)) & 1, abort, p.a.status, 8))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(tO + 128 * st + c, o);
                  tmem_wait16(o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st16(tO + 128 * st + c, o);
                }
              }
              l *= f;
              m = mnew;
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t neg = pack2(-mm, -mm);
            uint64_t sum[4] = {0, 0, 0, 0};  // (pairs of zeros)
#pragma unroll
            for (int c = 0; c < kW / 32; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int j = 32 * c + 2 * i;
                float2 x = unpack2(fma2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), scale2, neg));
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                sum[i & 3] = add2(sum[i & 3], pack2(x.x, x.y));
                pk[i] = pack_bf16(x.x, x.y);
              }
              tmem_st16(tSh + 16 * c, pk);
            }
            const float2 total = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
            l += total.x + total.y;
            tmem_wait_st();
            tc_fence_before();
          }
          mbar_arrive(bars.pready(st, h));
        }
        ++ns;
      }
      if (!ok) break;
      // ------------------------------------------------------------ the item's result
      const bool whole = nb == it.nblk;
      const int head = it.kvh * p.gs + (row - node_in * p.gs);
      uint16_t* const dst = static_cast<uint16_t*>(p.a.out) + it.b * p.a.out_stride[0] + node * p.a.out_stride[1] + head * p.a.out_stride[2];
      // partial results: first item of the run in slot 0, a later (so last) one in slot 1
      const int slot = u0 >= it.unit0 ? 0 : 1;
      const long long pt = ((long long)blockIdx.x * 2 + slot) * (TWO ? 2 : 1) + tile;
      float4* part = reinterpret_cast<float4*>(p.part) + pt * (HD / 4) * kBlk + row;
      float w0 = 1.f, w1 = 0.f;      // weights of the streams' sums (TWO: of this one's)
      bool other = false;            // stream 1 had a block (TWO = false)
      if (TWO) {
        if (!(ok = op_wait(bars.ofull(st), no[0]++ & 1, abort, p.a.status, 10))) break;
      } else {
        // The streams' rows lie in the same lanes: each warpgroup joins one half of the columns
        // of both sums.
        sh.ml[st][row] = make_float2(m, l);
        if (!(ok = meet())) break;
        const float2 a = sh.ml[0][row], b = sh.ml[1][row];
        m = fmaxf(a.x, b.x);
        const float mm = m == -INFINITY ? 0.f : m;
        w0 = ex2(a.x - mm);
        w1 = ex2(b.x - mm);
        l = a.y * w0 + b.y * w1;
        other = nb > 1;
        if (!(ok = op_wait(bars.ofull(0), no[0]++ & 1, abort, p.a.status, 10))) break;
        if (other && !(ok = op_wait(bars.ofull(1), no[1]++ & 1, abort, p.a.status, 11))) break;
      }
      tc_fence_after();
      const bool fix = *reinterpret_cast<volatile int*>(&sh.bad_v) != 0;
      const float mm = m == -INFINITY ? 0.f : m;
      if (!whole && node >= 0 && (TWO || st == 0)) p.part_ml[pt * kBlk + row] = make_float2(m, l);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (warp_live) {
        const int c0 = TWO ? 0 : (int)st * (HD / 2), c1 = TWO ? HD : c0 + HD / 2;
        const uint32_t own = tO + (TWO ? 128 * st : 0);
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          uint32_t u[16], v[16];
          float o[16];
          tmem_ld16(own + c, u);
          if (other) tmem_ld16(tO + 128 + c, v);
          tmem_wait16(u);
          tmem_wait16(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = __uint_as_float(u[i]);
            if (!TWO) o[i] = w0 * o[i] + (other ? w1 * __uint_as_float(v[i]) : 0.f);
          }
          if (node >= 0) put16(o, whole, inv, dst, part, c);
        }
        if (fix && node >= 0) put_nonfinite<HD>(p, it, r, head, mm, inv, c0, c1, whole ? dst : nullptr, part);
      }
      tc_fence_before();
      if (!TWO && !(ok = meet())) break;
    }
  } else {
    // (a walk in local memory costs 2000 cycles: what shared memory leaves of L1 does not hold it)
    Run& run = sh.runs[warp - 8];
    if (lane == 0) run = begin;
    __syncwarp();
    auto next = [&]() -> bool {
      bool more = false;
      __syncwarp();
      if (lane == 0) more = run.next(p);
      __syncwarp();
      return uniform(more);
    };
    if (warp == 8) {
      // ---------------------------------------------------------------- producer
      // lane i < 8 looks up page i of a block; the table is read two blocks ahead and not looked at
      // before it is needed, so that its latency is nobody's
      Ring put, block;                // ring slots; blocks
      uint32_t fill = 0, qphase = 0;  // ring slots filled; Q loads done
      bool ok = true;
      auto look_up = [&](const Item& it, int j) -> int {
        const int at = (it.kstart + j * kBlk) / kOpPage + lane;
        return lane < 8 && at * kOpPage < it.end ? op_ld(p.c.page_table + (long long)it.b * p.c.max_pages + at) : 0;
      };
      while (ok && next()) {
        const Item it = run.it;
        const int blocks = (int)uniform(it.jb - it.ja);
        const uint32_t rows = p.npt * p.gs;
        int page1 = look_up(it, it.ja), page2 = look_up(it, it.ja + 1);
        for (int blk = 0; ok && blk < blocks; ++blk) {
          const int j = it.ja + blk;
          const uint32_t live = uniform(min(kBlk / kOpPage, (it.end - it.kstart - j * kBlk + kOpPage - 1) / kOpPage));
          int page = page1;
          page1 = page2;
          page2 = look_up(it, j + 2);
          if (page < 0 || page >= p.c.n_pages) {
            op_error(p.a.status, MK_ERR_BAD_PAGE, it.b, (it.kstart + j * kBlk) / kOpPage + lane, page);
            page = 0;
          }
          __syncwarp();
          const int first = (page * p.c.n_kv_heads + it.kvh) * (kOpPage / 8);  // its first row group
          uint32_t group[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) group[i] = __shfl_sync(0xffffffffu, first, i);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++fill, put.advance(kStages)) {
            const uint32_t s = put.slot;
            if (!(ok = op_wait(bars.empty(s), put.phase ^ 1, abort, p.a.status, 1))) break;
            if (elect_one()) {
              const uint32_t dst = ring + s * C::kTile, bar = kv ? bars.vfull(block.slot) : bars.kfull(block.slot);
              mbar_expect_tx(bar, live * kOpPage * HD * 2);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (i < live) op_tma_4d(dst + i * (kOpPage * HD * 2), kv ? &tv : &tk, 0, 0, 0, (int)group[i], bar);
            }
            __syncwarp();
            if (kv == 0 && blk == 0) {  // the item's queries, once the last item's products have read theirs
              if (!(ok = op_wait(bars.qempty(), (qphase & 1) ^ 1, abort, p.a.status, 2))) break;
              ++qphase;
              const uint32_t tiles = uniform(TWO && (it.tp * 2 + 1) * p.npt < it.cnt ? 2 : 1);
              const int head = (int)uniform(it.kvh * p.gs), node = (int)uniform(it.tp * nodes_per_group(p)), seq = (int)uniform(it.b);
              if (elect_one()) {
                mbar_expect_tx(bars.qfull(), tiles * rows * HD * 2);
                for (uint32_t t = 0; t < tiles; ++t)
                  for (int h = 0; h < C::kHalves; ++h)
                    op_tma_4d(q_s + t * C::kTile + h * (kBlk * C::kSpan), &tq, h * (C::kSpan / 2), head,
                              node + (int)t * p.npt, seq, bars.qfull());
              }
              __syncwarp();
            }
          }
          block.advance(kStages);
        }
      }
      // an abandoned run leaves copies in flight: wait for them (bounded)
      if (*abort) {
        const uint32_t n = min(fill, kStages);
        for (uint32_t f = fill - n; f < fill; ++f)
          mbar_wait(f & 1 ? bars.vfull(f / 2 % kStages) : bars.kfull(f / 2 % kStages), (f / 2 / kStages) & 1, 10000000ll);
        if (qphase) mbar_wait(bars.qfull(), (qphase - 1) & 1, 10000000ll);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------------- products
      // Products execute in the order of their issue: S may be issued into a buffer as soon as the
      // P V that reads its old P is.  Queries: spans of 128 rows one behind the other (one copy
      // each); keys: see TreeCfg.
      constexpr int kW = kBlk / 2 * kParts;
      constexpr uint32_t idesc_s = umma_idesc_bf16(128, kW);
      constexpr uint32_t idesc_o = umma_idesc_bf16_bmn(128, HD);
      constexpr uint32_t kTileOff = C::kTile / 16;
      if (elect_one()) {
        const uint64_t dq = umma_sdesc_sw(q_s, 16, 8 * C::kSpan, C::kSpan), dk = umma_sdesc_sw(ring, 16, C::kGroup, C::kSpan);
        const uint64_t dv = umma_sdesc_sw(ring, 8 * C::kSpan, C::kGroup, C::kSpan);
        uint32_t nq = 0;                  // items
        bool ok = true;
        // S of half h (or all) of the K block in `slot`, done with it if `last`
        auto issue_s = [&](uint32_t st, uint32_t h, uint32_t slot, bool last) {
          const uint64_t a = dq + (TWO ? st : 0) * kTileOff, b = dk + slot * kTileOff + h * (kW / 8 * C::kGroup / 16);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = ((kk * 32 / C::kSpan) * (kBlk * C::kSpan) + (kk * 32) % C::kSpan) / 16;
            umma_bf16(tmem + kTmemS + 128 * st + kW * h, a + off, b + C::column16(kk) / 16, idesc_s, kk > 0);
          }
          umma_commit(bars.sfull(st, h));
          if (last) umma_commit(bars.empty(slot));
        };
        auto issue_pv = [&](uint32_t st, uint32_t h, uint32_t slot, bool first, bool last) {
          tc_fence_after();
          const uint64_t b = dv + slot * kTileOff + h * (kW / 8 * C::kGroup / 16);
          const uint32_t o = tmem + kTmemO + 128 * st, sp = tmem + kTmemS + 128 * st + kW * h;
#pragma unroll
          for (int kk = 0; kk < kW / 16; ++kk)
            umma_bf16_ta(o, sp + 8 * kk, b + kk * (2 * C::kGroup / 16), idesc_o, !first || kk > 0);
          if (!TWO) umma_commit(bars.pvdone(st, h));
          if (last) umma_commit(bars.empty(slot));
        };
        Ring ks, vs, kb;                  // slots of the next K and V block, and K's count
        vs.advance(kStages);
        uint32_t np[2] = {0, 0};          // blocks of the streams whose P V is issued
        Ring vst[2];                      // (TWO = false) the V slots of the streams' next blocks
        while (ok && run.next(p)) {
          const int nb = run.it.jb - run.it.ja;
          if (!(ok = op_wait1(bars.qfull(), nq++ & 1, abort, p.a.status, 3))) break;
          if (TWO) {
            auto next_s = [&](uint32_t st) {
              issue_s(st, 0, ks.slot, st == 1);
              if (st == 1) {
                ks.advance(kStages);
                ks.advance(kStages);
                kb.advance(kStages);
              }
            };
            if (!(ok = op_wait1(bars.kfull(kb.slot), kb.phase, abort, p.a.status, 4))) break;
            tc_fence_after();
            next_s(0);
            next_s(1);
            for (int blk = 0; ok && blk < nb; ++blk) {
              const uint32_t ph = np[0]++ & 1;
#pragma unroll
              for (uint32_t st = 0; st < 2; ++st) {
                // P is written, V clean and the next K there: see the cleaners
                if (!ok || !(ok = op_wait1(bars.pready(st, 0), ph, abort, p.a.status, 5))) break;
                issue_pv(st, 0, vs.slot, blk == 0, st == 1);
                if (blk + 1 < nb)
                  next_s(st);
                else
                  umma_commit(bars.ofull(st));
              }
              vs.advance(kStages);
              vs.advance(kStages);
            }
          } else {
            // whatever is ready: S by block and half, P V of either stream by its blocks and halves
            int qb = 0, pb[2] = {0, 1};
            uint32_t qh = 0, ph[2] = {0, 0};
            vst[0] = vst[1] = vs;
            vst[1].advance(kStages);
            vst[1].advance(kStages);
            uint64_t since = gtime();
            while (pb[0] < nb || pb[1] < nb) {
              bool moved = false;
              // (its buffer is free when the stream is past the block before, or past this half of it)
              const uint32_t qs = qb & 1;
              const int at = qs ? pb[1] : pb[0];
              if (qb < nb && (at == qb || (at + 2 == qb && (qs ? ph[1] : ph[0]) > qh)) &&
                  (qh == 1 || op_test(bars.kfull(kb.slot), kb.phase))) {
                tc_fence_after();
                issue_s(qs, qh, ks.slot, qh == 1);
                if (qh == 1) {
                  ks.advance(kStages);
                  ks.advance(kStages);
                  kb.advance(kStages);
                  ++qb;
                }
                qh ^= 1;
                moved = true;
              }
#pragma unroll
              for (uint32_t st = 0; st < 2; ++st) {
                if (pb[st] >= nb || !op_test(bars.pready(st, ph[st]), np[st] & 1)) continue;
                issue_pv(st, ph[st], vst[st].slot, pb[st] == (int)st && ph[st] == 0, ph[st] == 1);
                if (ph[st] == 1) {
                  if (pb[st] + 2 >= nb) umma_commit(bars.ofull(st));
                  pb[st] += 2;
                  ++np[st];
#pragma unroll
                  for (int i = 0; i < 4; ++i) vst[st].advance(kStages);
                }
                ph[st] ^= 1;
                moved = true;
              }
              if (moved) {
                since = gtime();
              } else if (*abort || (long long)(gtime() - since) > kOpWaitNs) {
                if (!*abort) op_error(p.a.status, MK_ERR_TIMEOUT, (int)blockIdx.x, 6, qb);
                *abort = 1;
                ok = false;
                break;
              }
            }
            // the next item's first V: behind this one's last
            for (int i = 0; i < (2 * nb) % (int)kStages; ++i) vs.advance(kStages);
          }
          if (ok) umma_commit(bars.qempty());
        }
      }
      __syncwarp();
      if (*abort) {  // let the products in flight end before the memory goes
        const uint64_t t0 = gtime();
        while ((long long)(gtime() - t0) < 10000000ll) {}
      }
    } else {
      // ---------------------------------------------------------------- cleaning
      // Arrives with a block's P on `pready` once its V is fit for use, at most one phase ahead.
      // (TWO: and once the next K is there, so that the product thread has one wait a step.)
      Ring at, block;       // V's ring slot, block
      at.advance(kStages);
      uint32_t n[2] = {0, 0};
      bool ok = true;
      auto arrive = [&](uint32_t st, uint32_t k) -> bool {
        if (k > 0 && !op_wait(bars.pready(st, 0), (k - 1) & 1, abort, p.a.status, 13)) return false;
        mbar_arrive(bars.pready(st, 0));
        return true;
      };
      while (ok && next()) {
        const Item it = run.it;
        const int nb = (int)uniform(it.jb - it.ja);
        for (int blk = 0; ok && blk < nb; ++blk) {
          const int k0 = it.kstart + (it.ja + blk) * kBlk;
          if (!(ok = op_wait(bars.vfull(block.slot), block.phase, abort, p.a.status, 12))) break;
          if (uniform(masked_block(p, it, k0))) {
            clean_v<HD, kCleaners>(ring_g + at.slot * C::kTile, it.end - k0, (int)threadIdx.x - (kTreeThreads - kCleaners), &sh.bad_v);
            fence_proxy_async_smem();
          }
          block.advance(kStages);
          at.advance(kStages);
          at.advance(kStages);
          if (TWO) {
            if (blk + 1 < nb && !(ok = op_wait(bars.kfull(block.slot), block.phase, abort, p.a.status, 14))) break;
            ok = arrive(0, n[0]++) && arrive(1, n[1]++);
          } else {
            ok = blk & 1 ? arrive(1, n[1]++) : arrive(0, n[0]++);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining the parts
// A block joins (row, 4 columns) pieces of one row tile of an item, rows side by side as the
// parts have them.  Few items have many parts each (38 at batch 1 with 4 KV heads): GROUPS = 4
// groups of threads share them and meet in shared memory, a piece per thread.  Many items have
// fewer than nine: GROUPS = 1, and four pieces per thread where that still leaves every SM its blocks.
// A block adds up a work list of up to 256 entries itself; the lengths are read behind the wait like
// everything else: that the first kernel's blocks had waited before they triggered makes them final, not
// visible to this kernel.  (Read in front of the wait they saved 1.2 us of the 12.7 that 8 nodes at 2K of one
// sequence take.)

template <int HD, int GROUPS, int PIECES>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ TreeParams p) {
  constexpr int kSide = kJoinThreads / GROUPS, kN = PIECES;
  __shared__ float4 s_o[GROUPS][kSide];
  __shared__ float2 s_ml[GROUPS][kSide];
  __shared__ int s_units[2][kJoinThreads / 32];
  const int tiles = p.two ? 2 : 1, rows = p.npt * p.gs;
  int i = blockIdx.x;
  const int tile = p.two ? i & 1 : 0;
  i = p.two ? i >> 1 : i;
  const int tp = i % p.ntp;
  i /= p.ntp;
  const int kvh = i % p.c.n_kv_heads, b = i / p.c.n_kv_heads;
  const int group = threadIdx.x / kSide, side = threadIdx.x % kSide;
  const int member = tp % p.team, e = b * p.groups + tp / p.team, E = num_entries(p);
  pdl_wait();
  pdl_trigger();
  const Entry x = make_entry(p, e, false);
  const int end = group_end(p, x.s, tp), nblk = (end - x.kstart + kBlk - 1) / kBlk;
  int row[kN], c4[kN];
  bool live[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int at = (blockIdx.y * kN + n) * kSide + side;
    c4[n] = at / rows;
    row[n] = at - c4[n] * rows;
    live[n] = c4[n] < HD / 4 && tp * nodes_per_group(p) + tile * p.npt + row[n] / p.gs < x.s.cnt;
  }
  int U = 0, before = 0;  // units of the list, and of the entries before this one
  if (E <= kJoinThreads) {
    if (threadIdx.x < E) U = make_entry(p, (int)threadIdx.x, false).units * p.c.n_kv_heads;
    if (threadIdx.x < e) before = U;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      U += __shfl_xor_sync(0xffffffffu, U, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    if ((threadIdx.x & 31) == 0) {
      s_units[0][threadIdx.x >> 5] = U;
      s_units[1][threadIdx.x >> 5] = before;
    }
    __syncthreads();
    U = before = 0;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      U += s_units[0][w];
      before += s_units[1][w];
    }
  } else {
    const int chunk = (E + kScan - 1) / kScan;
    for (int y = e / chunk * chunk; y < e; ++y) before += make_entry(p, y, false).units * p.c.n_kv_heads;
    U = op_ld(p.table + kScan);
    before += op_ld(p.table + e / chunk);
  }
  if (end == 0 || U <= 0) return;
  const int n_run = run_units(p, U), g0 = before + kvh * x.units;
  const int r0 = (g0 + kItemUnits) / n_run, r1 = (g0 + kItemUnits + nblk - 1) / n_run;
  if (r0 == r1) return;  // written whole
  // slot 0 holds the item that a run starts in: every part but, maybe, the first
  const int slot0 = r0 * n_run >= g0 ? 0 : 1;
  auto part_of = [&](int r) -> long long { return (((long long)r * p.team + member) * 2 + (r == r0 ? slot0 : 0)) * tiles + tile; };
  float m[kN], l[kN];
  float4 o[kN];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.f;
    o[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  constexpr int kBatch = PIECES > 1 ? 2 : 4;  // parts whose loads go out together
  for (int r = r0 + group; r <= r1; r += GROUPS * kBatch) {
    float2 ml[kBatch][kN];
    float4 y[kBatch][kN];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = min(r + k * GROUPS, r1);
      const long long pt = part_of(q);
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        ml[k][n] = make_float2(-INFINITY, 0.f);
        y[k][n] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live[n] && r + k * GROUPS <= r1) {
          ml[k][n] = p.part_ml[pt * kBlk + row[n]];
          const uint4 u = op_ld16_once(reinterpret_cast<const float4*>(p.part) + (pt * (HD / 4) + c4[n]) * kBlk + row[n]);
          y[k][n] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      float top = m[n];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k][n].x);
      const float mm = top == -INFINITY ? 0.f : top, f = ex2(m[n] - mm);
      m[n] = top;
      l[n] *= f;
      o[n] = make_float4(o[n].x * f, o[n].y * f, o[n].z * f, o[n].w * f);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = ex2(ml[k][n].x - mm);
        l[n] += w * ml[k][n].y;
        o[n].x += w * y[k][n].x;
        o[n].y += w * y[k][n].y;
        o[n].z += w * y[k][n].z;
        o[n].w += w * y[k][n].w;
      }
    }
  }
  if (GROUPS > 1) {
    s_o[group][side] = o[0];
    s_ml[group][side] = make_float2(m[0], l[0]);
    __syncthreads();
    if (group) return;
    float top = m[0];
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) top = fmaxf(top, s_ml[k][side].x);
    const float mm = top == -INFINITY ? 0.f : top;
    l[0] = 0.f;
    o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const float2 ml = s_ml[k][side];
      const float4 y = s_o[k][side];
      const float w = ex2(ml.x - mm);
      l[0] += w * ml.y;
      o[0].x += w * y.x;
      o[0].y += w * y.y;
      o[0].z += w * y.z;
      o[0].w += w * y.w;
    }
  }
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    if (!live[n]) continue;
    const float inv = l[n] == 0.f ? 0.f : 1.f / l[n];
    const int node = tp * nodes_per_group(p) + tile * p.npt + row[n] / p.gs;
    uint16_t* dst = static_cast<uint16_t*>(p.a.out) + b * p.a.out_stride[0] + node * p.a.out_stride[1] +
                    (long long)(kvh * p.gs + row[n] % p.gs) * p.a.out_stride[2] + 4 * c4[n];
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[n].x * inv, o[n].y * inv), pack_bf16(o[n].z * inv, o[n].w * inv));
  }
}

template <int HD, bool TWO>
cudaError_t launch_one(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(tree_kernel<HD, TWO>, TreeSmem<HD>::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_early(tree_kernel<HD, TWO>, dim3((unsigned)p.grid), kTreeThreads, TreeSmem<HD>::kBytes, st, p, tq, tk, tv);
}

template <int HD>
cudaError_t launch_hd(const TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      cudaStream_t st) {
  const cudaError_t e = p.two ? launch_one<HD, true>(p, tq, tk, tv, st) : launch_one<HD, false>(p, tq, tk, tv, st);
  if (e != cudaSuccess) return e;
  if (p.c.max_pages <= kBlk / kOpPage) return cudaSuccess;  // items of one block: nothing is split
  const long long heads = (long long)p.c.batch * p.c.n_kv_heads * p.ntp;
  // One group of threads where an item has up to 9 parts (512 nodes of 8 sequences 145 us, with four groups
  // 355; 16 nodes at 32K of 8 sequences 97.0, 103.4), four where it has more (one node at 8K of one sequence
  // 16.7 us, with one group 23.0).  Four pieces a thread where that leaves every SM four blocks (chunk of 2001 at
  // 8K 224 us, with one piece 240; prompt of 4096 155, 185), else one (8 ragged sequences of 16 nodes 58.0, with
  // four 60.5).
  const bool many = 8 * heads > p.grid;
  const long long all = heads * (p.two ? 2 : 1) * p.npt * p.gs * (HD / 4);  // pieces of all items
  const bool four = many && all > 4ll * kJoinThreads * p.grid * 4;
  const int pieces = four ? 4 * kJoinThreads : many ? kJoinThreads : kJoinThreads / 4;
  const dim3 grid((unsigned)(heads * (p.two ? 2 : 1)), (unsigned)((p.npt * p.gs * (HD / 4) + pieces - 1) / pieces));
  return launch_early(four ? join_kernel<HD, 1, 4> : many ? join_kernel<HD, 1, 1> : join_kernel<HD, 4, 1>, grid, kJoinThreads, 0, st, p);
}

}  // namespace

size_t tree_workspace_bytes(const TreeParams& p) {
  const size_t tiles = (size_t)p.grid * 2 * (p.two ? 2 : 1);
  return tiles * kBlk * ((size_t)p.c.head_dim * 4 + sizeof(float2)) + (kScan + 1) * sizeof(int);
}

cudaError_t launch_tree(TreeParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t st) {
  const size_t tiles = (size_t)p.grid * 2 * (p.two ? 2 : 1);
  p.part = static_cast<float*>(p.a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part + tiles * kBlk * p.c.head_dim);
  p.table = reinterpret_cast<int*>(p.part_ml + tiles * kBlk);
  if (p.c.head_dim == 128) return launch_hd<128>(p, tq, tk, tv, st);
  if (p.c.head_dim == 64) return launch_hd<64>(p, tq, tk, tv, st);
  return launch_hd<32>(p, tq, tk, tv, st);
}

}  // namespace mk
